"""The debug build's index checks and guard bands around 8-bit pages, rotations and rotated rows; the results are
those of the release build bit for bit."""
import numpy as np
import pytest

from test_gpu_kv_debug import Guards, debug_lib, ints, walk  # noqa: F401  (debug_lib: a fixture)
from transformer_layer_decode_gb300 import dec, kv, rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("hd,io,nkv,group,R", [
    (64, torch.float32, 2, 3, 16), (64, torch.bfloat16, 1, 12, 64), (128, torch.float32, 1, 8, 32),
    (128, torch.bfloat16, 3, 1, 128)])
def test_every_call_between_guards(debug_lib, hd, io, nkv, group, R):  # noqa: F811
    checked, guards = walk(debug_lib, "q8", hd, io, nkv, group, R)
    guards.check()
    plain, guards = walk(dec.LIB_PATH, "q8", hd, io, nkv, group, R)
    guards.check()
    assert len(checked) == len(plain)
    for i, (a, b) in enumerate(zip(checked, plain)):
        assert torch.equal(a, b) and not bool(torch.isnan(a.float()).any()), i


def rotated(lib_path, fmt, hd, rot, layout, io, nkv, heads, R, n):
    """Rotations and rotated rows on guarded memory; (everything they gave, the guards)."""
    g = Guards()
    gen = torch.Generator(device="cuda").manual_seed(hd + rot + n)
    n_seqs = max(3, n // 40)
    width = -(-(n // n_seqs + 21) // R)
    shape = kv.KVCacheDesc(1, nkv, hd, R, n_seqs * width, n_seqs, width, kv.FORMATS[fmt])
    page = kv.ctypes.c_size_t()
    assert dec.load_library(lib_path).dec_kv_sizes(kv.ctypes.byref(shape), kv.ctypes.byref(page), None) == 0
    c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, lib_path=lib_path,
                   pool=g.make((1, n_seqs * width, page.value), torch.uint8, 0),
                   table=g.make((n_seqs, width), torch.int32, -1), lens=g.make((n_seqs,), torch.int32, 0),
                   refs=g.make((n_seqs * width,), torch.int32, 1))
    c.table.copy_(ints(np.arange(n_seqs * width).reshape(n_seqs, width)))
    c.scratch, c.status = g.make((c.scratch.numel(),), torch.int32), g.make((1,), torch.int32, 0)
    c.desc.scratch, c.desc.status = c.scratch.data_ptr(), c.status.data_ptr()
    r = rope.Rotary(hd, rot_dim=rot, layout=layout, lib_path=lib_path)
    steps = g.make((rot // 2,), torch.int64)
    steps.copy_(r.steps)
    r.steps = steps
    r.desc.steps = steps.data_ptr()

    def given(*shape):
        t = g.make(shape, io)
        t.copy_(torch.randn(*shape, device="cuda", generator=gen))
        return t

    rng = np.random.default_rng(n)
    plan = [(t % n_seqs, t // n_seqs) for t in range(n)]
    order = rng.permutation(n)
    seqs = g.make((n,), torch.int32)
    positions = g.make((n,), torch.int32)
    seqs.copy_(ints([plan[i][0] for i in order]))
    positions.copy_(ints([plan[i][1] for i in order]))
    q, k, v, out = given(n, heads, hd), given(n, nkv, hd), given(n, nkv, hd), g.make((n, heads, hd), io, 0)
    c.append_rotated(0, r, q, k, v, seqs=seqs, positions=positions, q_out=out)
    seen = [out, r.rotate(k, positions, out=g.make((n, nkv, hd), io, 0)),
            r.rotate(q, positions, out=q, backward=True)]
    c.lens.copy_(ints([1 + max([p for s, p in plan if s == i], default=0) for i in range(n_seqs)]))
    c.extend()
    last = g.make((n_seqs, heads, hd), io, 0)
    c.append_rotated(0, r, given(n_seqs, heads, hd), given(n_seqs, nkv, hd), given(n_seqs, nkv, hd), q_out=last)
    c.sync_status()
    return seen + [last, c.pool], g


@pytest.mark.parametrize("fmt", ["q8", "q4", "bf16"])
@pytest.mark.parametrize("hd,rot,layout,io,nkv,heads,R,n", [
    (64, 64, "half", torch.float32, 1, 5, 16, 1), (128, 128, "half", torch.bfloat16, 3, 6, 48, 90),
    (128, 36, "half", torch.float32, 2, 2, 16, 700), (64, 24, "interleaved", torch.bfloat16, 5, 5, 32, 1111)])
def test_rotations_between_guards(debug_lib, fmt, hd, rot, layout, io, nkv, heads, R, n):  # noqa: F811
    checked, guards = rotated(debug_lib, fmt, hd, rot, layout, io, nkv, heads, R, n)
    guards.check()
    plain, guards = rotated(dec.LIB_PATH, fmt, hd, rot, layout, io, nkv, heads, R, n)
    guards.check()
    for i, (a, b) in enumerate(zip(checked, plain)):
        assert torch.equal(a, b), i
