"""Memory-safety checks of the paged cache that need no sanitizer (none can run here): the debug build of the
library, whose kernels check the indices of pages, rows, parts, lists and results before the access, with every
buffer between guard bands; the results are those of the release build bit for bit."""
import numpy as np
import pytest

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

GUARD, BYTE = 4096, 0xA5


@pytest.fixture(scope="module")
def debug_lib():
    return tld_build.build(debug=True)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


class Guards:
    def __init__(self):
        self.all = []

    def make(self, shape, dtype, fill=None):
        """A tensor between two guard bands; without a fill its bytes are the guards' too."""
        size = int(np.prod(shape)) * dtype.itemsize
        flat = torch.full((GUARD + -(-size // 16) * 16 + GUARD,), BYTE, dtype=torch.uint8, device="cuda")
        t = flat[GUARD:GUARD + size].view(dtype).view(shape)
        if fill is not None:
            t.fill_(fill)
        self.all.append((flat, size))
        return t

    def check(self):
        for flat, size in self.all:
            assert bool((flat[:GUARD] == BYTE).all()) and bool((flat[GUARD + size:] == BYTE).all()), size


def walk(lib_path, fmt, hd, io, nkv, group, R):
    """All calls, short and long, on guarded memory; (everything they gave, the guards)."""
    g = Guards()
    n_seqs, max_pages = 7, 2048 // R
    n_pages = 2 * max_pages
    shape = kv.KVCacheDesc(2, nkv, hd, R, n_pages, n_seqs, max_pages, kv.FORMATS[fmt])
    page = kv.ctypes.c_size_t()
    assert dec.load_library(lib_path).dec_kv_sizes(kv.ctypes.byref(shape), kv.ctypes.byref(page), None) == 0
    c = kv.KVCache(n_layers=2, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, lib_path=lib_path,
                   pool=g.make((2, n_pages, page.value), torch.uint8), table=g.make((n_seqs, max_pages), torch.int32, -1),
                   lens=g.make((n_seqs,), torch.int32, 0), refs=g.make((n_pages,), torch.int32, 0))
    c.scratch, c.status = g.make((c.scratch.numel(),), torch.int32), g.make((1,), torch.int32, 0)
    c.desc.scratch, c.desc.status = c.scratch.data_ptr(), c.status.data_ptr()
    gen = torch.Generator(device="cuda").manual_seed(hd + nkv)
    seen = []

    def given(*shape):
        t = g.make(shape, io)
        t.copy_(torch.randn(*shape, device="cuda", generator=gen))
        return t

    def fill(seqs, n):
        c.extend(ints(seqs), ints(n))
        s, p = ints(np.repeat(seqs, n)), ints(np.concatenate([np.arange(x) for x in n]))
        for layer in range(2):
            c.append(layer, given(sum(n), nkv, hd), given(sum(n), nkv, hd), seqs=s, positions=p)
        ko, vo = g.make((sum(n), nkv, hd), io), g.make((sum(n), nkv, hd), io)
        seen.extend(c.read(1, s, p, k_out=ko, v_out=vo))

    def attend(seqs, **kw):
        n = n_seqs if seqs is None else len(seqs)
        q, out = given(n, nkv * group, hd), g.make((n, nkv * group, hd), io, 0)
        ws = g.make((c.workspace().numel(),), torch.uint8)
        seen.append(c.attention(1, q, seqs=None if seqs is None else ints(seqs), out=out, workspace=ws, **kw))

    fill([0, 1, 3, 4], [1500, 1, R, 333])
    for seqs in (None, [0], [1], [4, -1, 0, 0], [3, 1, 4] * 60, [2], list(range(7)) * 40):
        attend(seqs)
        attend(seqs, window=70, sinks=5)
        attend(seqs, window=1000, sinks=16)
    c.fork(ints([4, 0, 3]), ints([5, 6, 2]))
    c.release(ints([0, 1]))
    c.compact()
    c.extend()
    c.append(0, given(n_seqs, nkv, hd), given(n_seqs, nkv, hd))
    c.append(1, given(n_seqs, nkv, hd), given(n_seqs, nkv, hd))
    attend(None)
    c.release(window=100, sinks=3)
    attend(None, window=100, sinks=3)
    c.release()
    c.sync_status()
    return seen + [c.table, c.refs, c.lens], g


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("hd,io,nkv,group,R", [
    (64, torch.float32, 2, 3, 16), (64, torch.bfloat16, 1, 12, 64), (128, torch.float32, 1, 8, 32),
    (128, torch.bfloat16, 3, 1, 128)])
def test_debug_build_with_guards(debug_lib, fmt, hd, io, nkv, group, R):
    checked, guards = walk(debug_lib, fmt, hd, io, nkv, group, R)
    guards.check()
    plain, guards = walk(dec.LIB_PATH, fmt, hd, io, nkv, group, R)
    guards.check()
    assert len(checked) == len(plain)
    for i, (a, b) in enumerate(zip(checked, plain)):
        assert torch.equal(a, b) and not bool(torch.isnan(a.float()).any()), i


@pytest.mark.parametrize("build", ["release", "debug"])
def test_a_failed_check_is_reported(debug_lib, build):
    """The status bit and the line beside it, as a kernel would leave them."""
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, n_pages=2, n_seqs=1, max_pages=1,
                   lib_path=debug_lib if build == "debug" else None)
    c.status.fill_(kv.DEC_KV_BAD_BOUNDS | kv.DEC_KV_BAD_INDEX)
    c.scratch[30] = 1234
    with pytest.raises(dec.DecError, match="line 1234.*0x9"):
        c.sync_status()
    c.sync_status()
