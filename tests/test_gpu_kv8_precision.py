"""Attention over 8-bit pages where rows all but cancel, against 64 bits."""
import numpy as np
import pytest

import kv8_reference as ref
from transformer_layer_decode_gb300 import kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hd,nkv,group", [(64, 1, 1), (64, 3, 8), (128, 2, 1), (128, 1, 12)])
@pytest.mark.parametrize("n", [2, 16, 40])
def test_weights_keep_22_bits(io, hd, nkv, group, n):
    """Rows in pairs whose values are x and -x and whose weights are 1 and e^-d, d = 0.9 * 2^-12: the output is
    x tanh(d / 2), about x * 2^-13.2.  (Weights of 11 bits are equal, and their output is 0.)  The scores are 0 and
    -d, a code of 1 times numbers of few bits and the scale: off by a few 2^-24 of d.  An exponential is good to 2^-20,
    a weight's two pieces to 2^-22, n weights are summed and n products accumulated in fp32: off by at most
    |x| * (2 * 2^-20 + 2^-22 + 2 * n * 2^-24), at n = 40 2^-16.9, and by half a step of the result's type."""
    R, d = 16, 0.9 * 2.0 ** -12
    pages, rng = ref.Pages8(nkv, hd, R), np.random.default_rng(n + hd)
    n_pages = -(-n // R)
    pool = np.zeros((1, n_pages, pages.page_bytes), np.uint8)
    x = rng.integers(1, 128, (nkv, hd)) * rng.choice([-1, 1], (nkv, hd))
    for i in range(n_pages):
        codes, scales = pages.parts(pool[0, i])
        codes[0][:] = 128
        codes[0][:, 1::2, 0] = 127
        codes[1][:, 0::2] = (128 + x)[:, None]
        codes[1][:, 1::2] = (128 - x)[:, None]
        for s in scales:
            s[:] = 1
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt="q8", pool=torch.from_numpy(pool).cuda(),
                   table=ints([list(range(n_pages))]), lens=ints([n]), refs=ints([1] * n_pages))
    q = torch.zeros(1, nkv * group, hd, device="cuda", dtype=io)
    q[..., 0] = 1
    scale = float(np.float32(d))
    got = c.attention(0, q, scale=scale)
    c.sync_status()
    got = got.double().cpu().numpy().reshape(nkv, group, hd)
    want = (x * np.tanh(scale / 2))[:, None]
    tol = np.abs(x)[:, None] * (2 * 2.0 ** -20 + 2.0 ** -22 + 2 * n * 2.0 ** -24 + scale * 2.0 ** -20)
    tol = tol + (np.abs(want) + tol) * torch.finfo(io).eps / 2
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
