"""The module that marshals a decode step's calls, on tensors of the GPU: what is plainly right it calls, once and with
these arguments; everything else it leaves to Python, whose answers and refusals are the same."""
import ctypes

import numpy as np
import pytest

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv, rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

CALLED = []
VP, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def stub(*types):
    f = ctypes.CFUNCTYPE(I32, *types)(lambda *a: CALLED.append(a) or 7)
    return f, ctypes.cast(f, VP).value


ROWS = stub(VP, I32, VP, VP, I32, I64, VP, VP, I32, VP)
ATTENTION = stub(VP, I32, VP, VP, I32, I64, I64, VP, I32, I32, I32, I32, F32, VP, SZ, VP)
ROTATED = stub(VP, I32, VP, VP, VP, I64, I64, I32, VP, VP, I32, I64, VP, VP, I32, VP)
ROTATE = stub(VP, VP, VP, I32, I64, I64, VP, I32, I32, I32, VP)
DESC, ROPE = 1 << 20, 1 << 21
N, HEADS, Q_HEADS, D = 5, 4, 8, 128


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def fast():
    tld_build.build()
    return dec.load_calls()


@pytest.fixture
def made(fast):
    """The module's contexts on stubs, and arguments that are right."""
    CALLED.clear()
    c = fast.context(DESC, 0, HEADS, D, ROWS[1], ROWS[1], ATTENTION[1], ROTATED[1])
    r = fast.context(ROPE, 0, 0, D, ROTATE[1])
    k, v = (torch.zeros(N, HEADS, D, device="cuda") for _ in range(2))
    q, out = (torch.zeros(N, Q_HEADS, D, device="cuda") for _ in range(2))
    return c, r, k, v, q, out, ints(range(N)), ints([3] * N)


def bad_rows(t):
    """What is not plainly rows like t."""
    wide = torch.zeros(t.shape[0], t.shape[1] + 1, 2 * t.shape[2], device="cuda", dtype=t.dtype)
    return {"on the CPU": t.cpu(), "half": t.half(), "double": t.double(), "a row less": t[1:], "flat": t.flatten(1),
            "another head_dim": t[..., :64].contiguous(), "not whole rows": wide[:, :-1, :t.shape[2]],
            "every second dimension": wide[:, :-1, ::2], "heads first": t.transpose(0, 1).contiguous().transpose(0, 1),
            "a list": t.tolist(), "none": None, "a number": 3, "sparse": t[:, 0].to_sparse(),
            "another type": t.bfloat16() if t.dtype == torch.float32 else t.float()}


def bad_list(t):
    return {"on the CPU": t.cpu(), "64 bits": t.long(), "an entry less": t[1:], "an entry more": torch.cat((t, t[:1])),
            "every second": t.repeat_interleave(2)[::2], "two-dimensional": t[None], "a list": t.tolist(), "bits": t.bool()}


BAD_INTS = {"negative": -1, "too large": 1 << 31, "far too large": 1 << 70, "a float": 1.0, "true": True, "none": None,
            "numpy's": np.int32(1)}


def vary(call, right, wrong):
    """call(*right) is made, and with any one argument changed to what `wrong` has for it nothing is."""
    assert call(*right) == 7 and len(CALLED) == 1
    for at, bads in wrong.items():
        for what, x in bads.items():
            args = list(right)
            args[at] = x
            assert call(*args) is None, (at, what)
    assert len(CALLED) == 1
    return CALLED.pop()


def test_rows(fast, made):
    c, _, k, v, _, _, seqs, pos = made
    stream = torch.cuda.current_stream().cuda_stream or None
    heads = {"a head less": k[:, 1:], "a head more": torch.zeros(N, HEADS + 1, D, device="cuda")}
    apart = torch.zeros(N, HEADS + 1, D, device="cuda")[:, :HEADS]
    wrong = {1: BAD_INTS, 2: bad_rows(k) | heads | {"another stride": apart}, 3: bad_rows(v) | heads | {"another stride": apart},
             4: bad_list(seqs), 5: bad_list(pos)}
    for call in (fast.append, fast.read):
        got = vary(call, [c, 1, k, v, seqs, pos], wrong)
        assert got == (DESC, 1, k.data_ptr(), v.data_ptr(), 0, HEADS * D, seqs.data_ptr(), pos.data_ptr(), N, stream)
        assert call(c, 0, apart, apart, seqs, None) == 7
        assert CALLED.pop() == (DESC, 0, apart.data_ptr(), apart.data_ptr(), 0, (HEADS + 1) * D, seqs.data_ptr(), None, N, stream)
        assert call(c, 0, k.bfloat16(), v.bfloat16(), seqs, None) == 7 and CALLED.pop()[4] == 1
    assert fast.append(c, 0, k, v, None, None) == 7 and CALLED.pop()[6:8] == (None, None)
    assert fast.read(c, 0, k, v, None, None) is None       # (without a list there is nothing to read)
    assert not CALLED


def test_attention(fast, made):
    c, _, _, _, q, out, seqs, _ = made
    stream = torch.cuda.current_stream().cuda_stream or None
    heads = {"a head less": q[:, 1:]}
    got = vary(fast.attention, [c, 1, q, out, seqs, 5, 2, 0.25, 1 << 22, 4096],
               {1: BAD_INTS, 2: bad_rows(q) | heads, 3: bad_rows(out) | heads, 4: bad_list(seqs), 5: BAD_INTS, 6: BAD_INTS,
                7: {"whole": 1, "none": None}, 8: {"none": None, "too large": 1 << 70}, 9: {"negative": -1, "none": None}})
    assert got == (DESC, 1, q.data_ptr(), out.data_ptr(), 0, Q_HEADS * D, Q_HEADS * D, seqs.data_ptr(), N, Q_HEADS, 5, 2, 0.25,
                   1 << 22, 4096, stream)


def test_rotated_rows(fast, made):
    c, r, k, v, q, out, seqs, pos = made
    stream = torch.cuda.current_stream().cuda_stream or None
    elsewhere = fast.context(ROPE, 1, 0, D, ROTATE[1])
    got = vary(fast.append_rotated, [c, 1, k, v, seqs, pos, r, q, out],
               {1: BAD_INTS, 2: bad_rows(k), 3: bad_rows(v), 4: bad_list(seqs), 5: bad_list(pos),
                6: {"none": None, "a number": 3, "of another device": elsewhere},
                7: {k: x for k, x in bad_rows(q).items() if k != "none"}, 8: bad_rows(out) | {"a head less": out[:, 1:]}})
    assert got == (DESC, 1, ROPE, q.data_ptr(), out.data_ptr(), Q_HEADS * D, Q_HEADS * D, Q_HEADS, k.data_ptr(), v.data_ptr(), 0,
                   HEADS * D, seqs.data_ptr(), pos.data_ptr(), N, stream)
    assert fast.append_rotated(c, 1, k, v, seqs, pos, r, None, None) == 7 and CALLED.pop()[3:8] == (None, None, 0, 0, 0)


def test_rotations(fast, made):
    _, r, _, _, q, out, _, pos = made
    stream = torch.cuda.current_stream().cuda_stream or None
    got = vary(fast.rotate, [r, q, pos, out, True],
               {1: bad_rows(q) | {"no heads": q[:, :0]}, 2: bad_list(pos), 3: bad_rows(out) | {"a head less": out[:, 1:]},
                4: {"a number": 1, "none": None}})
    assert got == (ROPE, q.data_ptr(), out.data_ptr(), 0, Q_HEADS * D, Q_HEADS * D, pos.data_ptr(), N, Q_HEADS, 1, stream)
    assert fast.rotate(r, q, None, out, False) == 7 and CALLED.pop()[6:] == (None, N, Q_HEADS, 0, stream)


def test_streams_and_devices(fast, made):
    c, r, k, v, q, out, seqs, pos = made
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert fast.append(c, 0, k, v, seqs, pos) == 7 and CALLED.pop()[-1] == side.cuda_stream
        assert fast.rotate(r, q, pos, out, False) == 7 and CALLED.pop()[-1] == side.cuda_stream
    there = fast.context(DESC, 1, HEADS, D, ROWS[1], ROWS[1], ATTENTION[1], ROTATED[1])  # (not the current device)
    assert fast.append(there, 0, k, v, seqs, pos) is None and not CALLED


# ---- both ways -------------------------------------------------------------------


class Counted:
    """The module, and how many of its calls it made."""

    def __init__(self, fast):
        self.fast, self.made, self.left = fast, 0, 0

    def __getattr__(self, name):
        def call(*args):
            rc = getattr(self.fast, name)(*args)
            self.made, self.left = self.made + (rc is not None), self.left + (rc is None)
            return rc
        return call


def caches(fast, fmt):
    out = []
    for way in (Counted(fast), None):
        c = kv.KVCache(n_layers=2, n_kv_heads=HEADS, head_dim=D, page_rows=16, fmt=fmt, n_pages=20, n_seqs=N, max_pages=4)
        c.pool.zero_()
        r = rope.Rotary(D)
        c.extend(n_new=ints([40, 1, 17, 33, 20]))
        if way is None:
            c._context = c._fast = r._context = r._fast = None
        else:
            c._fast = r._fast = way
        out.append((c, r, way))
    return out


@pytest.mark.parametrize("fmt", ["bf16", "q4", "q8"])
def test_a_step_goes_this_way_and_gives_the_same(fast, fmt):
    gen = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(N, Q_HEADS, D, device="cuda", generator=gen)
    k, v = (torch.randn(N, HEADS, D, device="cuda", generator=gen) for _ in range(2))
    seqs, pos, seen, ways = ints(range(N)), ints([39, 0, 16, 32, 19]), [], []
    for c, r, way in caches(fast, fmt):
        out, turned, rotated = (torch.zeros_like(q) for _ in range(3))
        kk, vv = torch.zeros_like(k), torch.zeros_like(v)
        c.append(0, k, v, seqs=seqs, positions=pos)
        c.append(1, k, v)
        c.append_rotated(1, r, q, k, v, q_out=turned)
        c.append_rotated(0, r, None, k, v, seqs=seqs)
        c.read(1, seqs, pos, k_out=kk, v_out=vv)
        c.attention(1, turned, out=out, window=9, sinks=1)
        r.rotate(q, pos, out=rotated, backward=True)
        c.sync_status()
        seen.append((c.pool, out, turned, rotated, kk, vv))
        ways.append(way)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    assert ways[0].made == 7 and ways[0].left == 0


def outcome(f):
    try:
        f()
    except Exception as e:  # noqa: BLE001
        return type(e), str(e)
    return None


def test_refusals_are_the_same(fast):
    (a, ra, way), (b, rb, _) = caches(fast, "q8")
    q, k = torch.zeros(N, Q_HEADS, D, device="cuda"), torch.zeros(N, HEADS, D, device="cuda")
    seqs = ints(range(N))
    odd = torch.zeros(1 + N * HEADS * D, device="cuda")[1:].view(N, HEADS, D)
    bads = list(bad_rows(k).items()) + [("unaligned", odd)]
    for c, what, make in [
            *((1, w, lambda c, r, x=x: c.append(0, x, k)) for w, x in bads if w not in ("none", "a list", "a number")),
            *((1, w, lambda c, r, x=x: c.append(0, k, k, seqs=x)) for w, x in bad_list(seqs).items() if w != "a list"),
            *((1, w, lambda c, r, x=x: c.append(x, k, k)) for w, x in (("layer", 2), ("layer", -1), ("layer", 1 << 31))),
            (1, "k over v", lambda c, r: c.read(0, seqs, k_out=k, v_out=k)),
            (1, "o over q", lambda c, r: c.attention(0, q, out=q)),
            (1, "heads", lambda c, r: c.attention(0, q[:, :6].contiguous(), out=q[:, :6].contiguous())),
            (1, "window", lambda c, r: c.attention(0, q, out=q.clone(), window=-1)),
            (1, "scale", lambda c, r: c.attention(0, q, out=q.clone(), scale=float("inf"))),
            (1, "workspace", lambda c, r: c.attention(0, q, out=q.clone(), workspace=q[:0])),
            (1, "q_out over k", lambda c, r: c.append_rotated(0, r, k, k.clone(), k.clone(), q_out=odd)),
            (1, "x over out", lambda c, r: r.rotate(q[1:], out=q[:-1])),
            (1, "positions", lambda c, r: r.rotate(q, seqs[1:], out=q))]:
        one, other = outcome(lambda: make(a, ra)), outcome(lambda: make(b, rb))
        assert one is not None and one == other, (what, one, other)
    for c in (a, b):
        c.sync_status()


def test_a_cache_without_the_module(monkeypatch):
    monkeypatch.setattr(dec, "load_calls", lambda: None)
    c = kv.KVCache(n_layers=1, n_kv_heads=HEADS, head_dim=D, fmt="bf16", n_pages=4, n_seqs=2, max_pages=1)
    r = rope.Rotary(D)
    c.extend()
    k = torch.ones(2, HEADS, D, device="cuda")
    out, q = torch.zeros(2, Q_HEADS, D, device="cuda"), torch.ones(2, Q_HEADS, D, device="cuda")
    assert c.append_rotated(0, r, q, k, k, q_out=out) is out and torch.equal(out, r.rotate(q, ints([0, 0])))
    assert torch.equal(c.attention(0, q, out=out), torch.ones_like(out))
    assert torch.equal(r.rotate(q, out=out), r.rotate(q))
    c.sync_status()
