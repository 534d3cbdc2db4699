"""Attention over 4-bit pages where the rows' weights and the blocks' values differ by many powers of two,
against 64 bits."""
import numpy as np
import pytest

from transformer_layer_decode_gb300 import kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

HEADS = 4


def dominant_and_tail(hd, n, drop, sizes, io, first=0.0, outlier=None):
    """Errors of the outputs, per block of 32 dimensions relative to the block's outputs: row 0 has the
    weight 1 and values `first` times as large as the others', every other row the weight 2^-drop; the values
    of block b are of the size sizes[b].  outlier: (row, block, factor) makes one row's block larger.
    Scores are exact (one product of numbers of a few bits) but for the scale's rounding and one more."""
    gen = torch.Generator(device="cuda").manual_seed(hd + drop)
    R = 64
    c = kv.KVCache(n_layers=1, n_kv_heads=HEADS, head_dim=hd, page_rows=R, fmt="q4", n_pages=-(-n // R), n_seqs=1,
                   max_pages=-(-n // R))
    c.extend(n_new=torch.tensor([n], dtype=torch.int32, device="cuda"))
    seqs, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    k = torch.zeros(n, HEADS, hd, device="cuda")
    k[0, :, 0] = 1.75
    v = torch.randn(n, HEADS, hd, device="cuda", generator=gen)
    v *= torch.tensor(sizes, device="cuda").repeat_interleave(32)
    v[0] *= first
    if outlier:
        row, block, factor = outlier
        v[row, :, 32 * block:32 * block + 32] *= factor
    c.append(0, k, v, seqs=seqs, positions=pos)
    _, v = c.read(0, seqs, pos)
    q = torch.zeros(1, HEADS, hd, device="cuda")
    q[..., 0] = 1
    scale = float(np.float32(drop * np.log(2) / 1.75))
    got = c.attention(0, q.to(io), scale=scale).double()
    c.sync_status()
    w = torch.full((n, 1, 1), float(np.exp(-1.75 * scale)), dtype=torch.float64, device="cuda")
    w[0] = 1
    want = (w * v.double()).sum(0, keepdim=True) / w.sum()
    norm = lambda x: x.unflatten(-1, (hd // 32, 32)).square().sum((0, 1, 3)).sqrt()  # noqa: E731
    return (norm(got - want) / norm(want)).tolist()


CASES = [  # sizes of the values by block, the first row's, one larger block of a row that hardly weighs
    ((1, 1, 1, 1), 0.0, None),
    ((1, 2.0 ** -10, 2.0 ** -14, 2.0 ** -18), 0.0, None),
    ((2.0 ** -18, 0.3, 1e3, 1), 0.0, None),
    ((1e3, 1, 1e-3, 1), 1e-3, None),
    ((1, 1, 1, 1), 0.0, (15000, 1, 4096.0)),
    ((1, 1e-3, 1, 1), 0.0, (3, 0, 4096.0)),
]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("sizes,first,outlier", CASES)
def test_fp32_results_keep_22_bits_of_every_block(hd, sizes, first, outlier):
    """Tail weights of 2^-20.  The score of 20 in log2 units takes three roundings (scale, product, difference
    from the reference) of 2^-24 each, 20 * 3 * 2^-24 * ln 2 = 2.5e-6, all rows alike; the exponential 2^-22,
    2.4e-7; the weights' pieces at most as much; sums over a few tiles a warp, rounded to the nearest, below
    1e-7.  (One power of two for all blocks and a second piece that meets fp16's smallest step: 1e-5 to 8e-2.)"""
    errors = dominant_and_tail(hd, 24000, 20, sizes[:hd // 32], torch.float32, first, outlier)
    assert max(errors) <= 3.1e-6, errors


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("sizes,first,outlier", CASES)
def test_bf16_results_keep_11_bits_of_every_block(hd, sizes, first, outlier):
    """As root mean squares: the results' own rounding, 2^-8 / sqrt(3) at most, 2.26e-3; a weight and its product
    with a scale, 2^-11 / sqrt(3) each, random from row to row like the values, 4e-4; where the scales are 2^-20,
    products near 2^-16 with a step of 2^-24: 2^-9.3 / sqrt(3), 9e-4.  2.5e-3 together.  The block that has
    the larger row keeps fewer bits of the others and is left out."""
    errors = dominant_and_tail(hd, 24000, 20, sizes[:hd // 32], torch.bfloat16, first, outlier)
    if outlier:
        del errors[outlier[1]]
    assert max(errors) <= 2.6e-3, errors
