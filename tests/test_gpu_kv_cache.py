"""The paged cache's operators on the GPU against their 64-bit statements.

Tolerances of attention.  A score is a sum of d products in fp32 (d + 8
roundings of 2^-24 relative to sum |q||k|, the scale and the split of q among
them), a weight is an exponential good to 2^-20, n weights are summed and n
products accumulated in fp32 (n * 2^-24 each at the very worst).  So an output
is off by at most sum_j w_j |v_j| * (2 * ds + 2 * n * 2^-24 + 2^-19), plus half
a step of its own type (bf16 2^-8, fp32 2^-24).

Over 4-bit pages a weight times its V scale enters as fp16 numbers: for fp32
results in two pieces, for bf16 results as one, so there the weight, and its
product with the scale, are each off by up to half a step of fp16, 2^-11: the
output by sum_j w_j |v_j| * 2^-10.  These numbers also have a smallest step:
they are off by at most 2^-25, where the weight that sets the reference is 2^9
and the scale enters as s / 2^e, 2^e <= 2 s for the largest scale s (of 2^-14 or
more).  With codes up to 8 and a sum of weights of at least 2^9, n rows are off
by at most n * 8 * 2^-25 / 2^9 * 2^e <= n * 2^-30 * s.  (For bf16 results scales
between 2^-7 and 1 enter as they are, e = 0, so there s counts as at least 1/2.)
It shows only where the rows that hold the weight are zero in a dimension.  A
block's largest code is 7, so s is the largest |v| / 7.
"""
import numpy as np
import pytest

import kv_reference as ref
from transformer_layer_decode_gb300 import dec, kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


def f32(t):
    return t.detach().float().cpu().numpy()


class Filled:
    """A cache whose sequences have the given lengths, its pool random bits where no row lies (NaN among
    them) and random rows elsewhere, at shuffled pages."""

    def __init__(self, fmt, nkv, hd, R, lens, *, layers=2, layer=1, seed=0, window=0, sinks=0, spare=3,
                 k_of=None, v_of=None, room=1):
        rng = np.random.default_rng(seed)
        self.pages = ref.Pages(fmt, nkv, hd, R)
        self.lens, self.layer, self.R = list(lens), layer, R
        width = max(-(-room // R), max(-(-n // R) for n in lens))
        table = np.full((len(lens), width), -1, np.int32)
        seen = [ref.visible(n, window, sinks) for n in lens]
        wanted = [(s, i) for s, v in enumerate(seen) for i in np.unique(v // R)]
        order = rng.permutation(len(wanted) + spare)
        for (s, i), p in zip(wanted, order):
            table[s, i] = p
        n_pages = len(order)
        pool = rng.integers(0, 256, (layers, n_pages, self.pages.page_bytes)).astype(np.uint8)
        if fmt == "bf16":   # NaN in every other place
            pool.view(np.uint16)[..., ::2] = 0x7FC0
        self.k, self.v = [], []
        for s, v in enumerate(seen):
            kk, vv = np.zeros((nkv, len(v), hd)), np.zeros((nkv, len(v), hd))
            for j, pos in enumerate(v):
                page = pool[layer, table[s, pos // R]]
                for h in range(nkv):
                    x = rng.normal(0, 1, hd) if k_of is None else k_of(s, h, pos, rng)
                    self.pages.put(page, 0, h, pos % R, x.astype(np.float32))
                    y = rng.normal(0, 1, hd) if v_of is None else v_of(s, h, pos, rng)
                    self.pages.put(page, 1, h, pos % R, y.astype(np.float32))
            vals = {p: self.pages.values(pool[layer, p]) for p in np.unique(table[s][table[s] >= 0])}
            for j, pos in enumerate(v):
                both = vals[table[s, pos // R]][:, :, pos % R]
                kk[:, j], vv[:, j] = both
            self.k.append(kk)
            self.v.append(vv)
        refs = np.bincount(table[table >= 0], minlength=n_pages)
        self.cache = kv.KVCache(n_layers=layers, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt,
                                pool=torch.from_numpy(pool).cuda(), table=ints(table), lens=ints(lens),
                                refs=ints(refs))

    def check(self, q, got, seqs, scale=None, what=""):
        scale = self.pages.d ** -0.5 if scale is None else scale
        bf16 = got.dtype == torch.bfloat16
        q, got = f32(q).astype(np.float64), f32(got).astype(np.float64)
        assert np.isfinite(got).all(), what
        for r, s in enumerate(seqs):
            if s < 0:
                continue
            o, size, dots = ref.attention(q[r], self.k[s], self.v[s], scale)
            n = self.k[s].shape[1]
            ds = (self.pages.d + 8) * 2.0 ** -24 * np.abs(dots)[:, None]
            tol = size * (2 * ds + 2 * n * 2.0 ** -24 + 2.0 ** -19)
            if self.pages.fmt == "q4" and n:
                top = np.abs(self.v[s]).max() / 7
                tol = tol + n * 2.0 ** -30 * max(top, 0.5 if bf16 and top > 2 ** -8 else 2 ** -14)
                tol = tol + (size * 2.0 ** -10 if bf16 else 0)
            tol = tol + (np.abs(o) + tol) * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-37
            bad = np.abs(got[r] - o) > tol
            assert not bad.any(), (what, r, s, n, np.argwhere(bad)[:4].tolist(), np.abs(got[r] - o)[bad][:4], tol[bad][:4])


SHAPES = [  # kv heads, group, head_dim, page rows
    (2, 4, 64, 128), (1, 1, 128, 16), (3, 2, 128, 64), (2, 8, 128, 32), (1, 12, 64, 48), (4, 3, 64, 16), (2, 5, 128, 128),
]


@pytest.mark.parametrize("room", [1, 40000])  # rows that a table has room for: short ones are not cut between CTAs
@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nkv,group,hd,R", SHAPES)
def test_attention_all_rows(fmt, io, nkv, group, hd, R, room):
    lens = [0, 1, 15, R, R + 1, 2 * R - 1, 333, 2]
    f = Filled(fmt, nkv, hd, R, lens, seed=nkv * 100 + hd + R, room=room)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(len(lens), nkv * group, hd, device="cuda", generator=g).to(io)
    out = f.cache.attention(f.layer, q)
    f.cache.sync_status()
    f.check(q, out, range(len(lens)))
    assert torch.all(out[0] == 0)                      # no rows: zeros
    again = f.cache.attention(f.layer, q)
    assert torch.equal(out, again)                     # the same bits


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (50, 3), (64, 200), (333, 1), (1000, 5),
                                          (100, 0), (2147483647, 2147483647)])
def test_attention_window_and_first_rows(fmt, window, sinks):
    lens = [0, 1, 2, 16, 31, 64, 100, 333, 517]
    f = Filled(fmt, 2, 64, 16, lens, seed=window % 1000 + sinks % 1000, window=window, sinks=sinks)
    q = torch.randn(len(lens), 6, 64, device="cuda")
    out = f.cache.attention(f.layer, q, window=window, sinks=sinks)
    f.cache.sync_status()
    f.check(q, out, range(len(lens)))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_long_sequences_and_rising_scores(fmt, hd):
    """Rows split over the whole GPU; scores that climb by 20 every 100 rows move the running maximum again
    and again, and the large values sit where the weights are small."""
    def k_of(s, h, pos, rng):
        x = rng.normal(0, 1, hd)
        return x if s else x * 0.01 + (pos % 1000) / 100 * 20 / hd ** 0.5

    def v_of(s, h, pos, rng):
        return rng.normal(0, 1, hd) * (100 if pos % 7 == 0 else 1)

    lens = [5003, 3001, 17]
    f = Filled(fmt, 1, hd, 64, lens, seed=hd, k_of=k_of, v_of=v_of)
    q = torch.randn(3, 4, hd, device="cuda")
    q[0] = 1.0
    out = f.cache.attention(f.layer, q)
    f.cache.sync_status()
    f.check(q, out, range(3))
    one = f.cache.attention(f.layer, q[:1].contiguous(), seqs=ints([0]))
    f.check(q[:1], one, [0])


@pytest.mark.parametrize("fmt,nkv,io,n", [
    ("bf16", 1, torch.float32, 140), ("q4", 1, torch.float32, 140), ("bf16", 2, torch.bfloat16, 300),
    ("q4", 2, torch.bfloat16, 300), ("q4", 3, torch.float32, 700)])
def test_attention_many_queries(fmt, nkv, io, n):
    """More queries than are counted at once, fewer and more units than CTAs, long and short and empty
    sequences and padding among them; with and without the last query of each."""
    lens = [0, 1, 40, 300, 4000, 17]
    f = Filled(fmt, nkv, 64, 32, lens, seed=n)
    rng = np.random.default_rng(n)
    seqs = rng.choice([-1, 0, 1, 2, 3, 5, 1, 2, 5], n)
    seqs[[3, n // 2, n - 2]] = 4
    q = torch.randn(n, 2 * nkv, 64, device="cuda").to(io)
    out = f.cache.attention(f.layer, q, seqs=ints(seqs))
    f.cache.sync_status()
    f.check(q, out, seqs)
    assert torch.all(out[torch.tensor(seqs < 1)] == 0)
    seqs[:] = rng.choice([1, 2], n)                      # all short, and hardly any
    out = f.cache.attention(f.layer, q, seqs=ints(seqs))
    f.check(q, out, seqs)
    seqs[:] = -1
    keep = torch.full_like(q, 3)
    assert torch.all(f.cache.attention(f.layer, q, seqs=ints(seqs), out=keep) == 3)
    seqs[n - 1] = 4
    out = f.cache.attention(f.layer, q, seqs=ints(seqs))
    f.check(q, out, seqs)
    f.cache.sync_status()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_lists_strides_and_padding(fmt):
    """Sequences in any order and twice, padding left as it was, q and out as parts of wider rows."""
    f = Filled(fmt, 2, 128, 32, [40, 70, 0, 200], seed=4)
    seqs = [3, -1, 1, 1, 0, -7, 2]
    wide = torch.randn(len(seqs), 4 * 128 + 512, device="cuda")
    q = wide[:, 128:128 + 512].unflatten(1, (4, 128))
    big = torch.full((len(seqs), 1024), 7.0, device="cuda")
    out = big[:, 256:768].unflatten(1, (4, 128))
    got = f.cache.attention(f.layer, q, seqs=ints(seqs), out=out, scale=0.25)
    f.cache.sync_status()
    assert got is out
    f.check(q, out, seqs, scale=0.25)
    assert torch.all(big[:, :256] == 7) and torch.all(big[:, 768:] == 7)
    assert torch.all(out[1] == 7) and torch.all(out[5] == 7)
    fresh = f.cache.attention(f.layer, q, seqs=ints(seqs), scale=0.25)
    assert torch.all(fresh[1] == 0) and torch.equal(fresh[0], out[0])
    # q and out side by side in the same rows
    both = torch.randn(4, 1024, device="cuda")
    q2 = both[:, :512].unflatten(1, (4, 128))
    keep = q2.clone()
    o2 = f.cache.attention(f.layer, q2, out=both[:, 512:].unflatten(1, (4, 128)))
    f.check(keep, o2, range(4))
    with pytest.raises(dec.DecError):
        f.cache.attention(f.layer, q2, out=both[:, 256:768].unflatten(1, (4, 128)))
    assert f.cache.attention(f.layer, q[:0], seqs=ints([])).shape == (0, 4, 128)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_extreme_queries(fmt):
    """Queries far above and below one, single large dimensions, zeros, a negative scale."""
    f = Filled(fmt, 1, 64, 16, [50, 50, 50, 50, 50], seed=9)
    q = torch.randn(5, 2, 64, device="cuda")
    q[0] *= 1e-30
    q[1] *= 2e4
    q[2] = 0
    q[3, :, 5] = 3e3
    q[4, 0] *= 1e-6
    for scale in (0.125, -0.02):
        out = f.cache.attention(f.layer, q, scale=scale)
        f.check(q, out, range(5), scale=scale)
    f.cache.sync_status()


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [(1e5,), (1e-3,), (3e-6,), (1e-4, 1, 1e4), (1e4, 1, 1e-4)])
def test_attention_value_sizes_over_4_bits(io, sizes):
    """V scales from fp16's smallest numbers to its largest, rising and falling along a sequence."""
    def v_of(s, h, pos, rng):
        return rng.normal(0, 1, 128) * sizes[pos * len(sizes) // 400]

    f = Filled("q4", 1, 128, 32, [400, 130], seed=12, v_of=v_of)
    q = torch.randn(2, 3, 128, device="cuda").to(io)
    out = f.cache.attention(f.layer, q)
    f.check(q, out, range(2), what=str(sizes))
    f.cache.sync_status()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_bad_pages_are_left_out(fmt):
    f = Filled(fmt, 1, 64, 16, [64, 64, 30], seed=5)
    q = torch.randn(3, 2, 64, device="cuda")
    f.cache.table[0, 2] = -1
    f.cache.table[1, 0] = 1 << 20
    out = f.cache.attention(f.layer, q)
    with pytest.raises(dec.DecError) as e:
        f.cache.sync_status()
    assert e.value.code == dec.DEC_ERR_DEVICE and "index" in str(e.value)
    f.cache.sync_status()                                # cleared
    for s, rows in ((0, [j for j in range(64) if not 32 <= j < 48]), (1, list(range(16, 64)))):
        f.k[s], f.v[s] = f.k[s][:, rows], f.v[s][:, rows]
    f.check(q, out, range(3))
    # sequences and lengths out of range: skipped
    f.cache.lens[0] = 65
    f.cache.lens[1] = -3
    keep = torch.full((4, 2, 64), 5.0, device="cuda")
    out = f.cache.attention(f.layer, torch.cat((q, q[:1])), seqs=ints([0, 1, 2, 3]), out=keep)
    with pytest.raises(dec.DecError):
        f.cache.sync_status()
    assert torch.all(out[[0, 1, 3]] == 5)
    f.check(q[2:], out[2:3], [2])


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_long_batch_does_not_drift(fmt):
    """Values that are all 0.875 (a 4-bit block's code 7 at scale 2^-3): the result is 0.875 whatever the
    weights are.  A warp takes T tiles of 16 rows one after another; its sums take T roundings for a
    value and 4 T for the weights' sum in a thread, each to the nearest and so without a direction, of a
    standard deviation of at most 2^-24 / sqrt(3) of the sum.  The results' errors have a root mean square
    of at most sqrt(5 T / 3) 2^-24, and 2^-22 for the weights' pieces and the last roundings.  (Sums that are
    cut off instead fall short by T 2^-25 and more, 1.2e-5 here.)"""
    n, seqs, heads, hd, R = 24000, 24, 16, 128, 64
    torch.manual_seed(0)
    c = kv.KVCache(n_layers=1, n_kv_heads=heads, head_dim=hd, page_rows=R, fmt=fmt, n_pages=n // R,
                   n_seqs=seqs, max_pages=n // R)
    c.table.copy_(torch.randperm(n // R, dtype=torch.int32, device="cuda").expand(seqs, -1))
    k = torch.randn(n, heads, hd, device="cuda")
    c.append(0, k, torch.full_like(k, 0.875), seqs=torch.zeros(n, dtype=torch.int32, device="cuda"),
             positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    c.lens.fill_(n)
    got = c.attention(0, torch.randn(seqs, heads, hd, device="cuda")).double()
    c.sync_status()
    warps = 12 * torch.cuda.get_device_properties(0).multi_processor_count
    tiles = seqs * heads * n / 16 / warps
    rms = ((got / 0.875 - 1) ** 2).mean().sqrt().item()
    assert rms <= (5 * tiles / 3) ** 0.5 * 2.0 ** -24 + 2.0 ** -22, rms


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_scores_keep_fp32(fmt, hd):
    """Scores of a standard deviation of 4, fp32 results.  A score's errors, as root mean squares: q in pieces
    of 22 bits, 2^-23 / sqrt(3) of each of its products and so of the score, 2.8e-7; five roundings of 2^-24
    of a block's sum (below 4), 2e-7; the score in log2 units (of 6) and its difference from the reference,
    2^-24 each, 4e-7; the exponential, 2^-22 / sqrt(3), 1.4e-7: 5.5e-7 together.  With values of mean 0 the
    outputs are off by as much of their own size.  (Codes as subnormal numbers: 1.2e-6 to 1.4e-6.)"""
    n, seqs, heads = 31, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(3)
    c = kv.KVCache(n_layers=1, n_kv_heads=heads, head_dim=hd, page_rows=16, fmt=fmt, n_pages=2 * seqs, n_seqs=seqs,
                   max_pages=2)
    c.extend(None, ints([n] * seqs))
    at, pos = ints(np.repeat(range(seqs), n)), ints(np.tile(range(n), seqs))
    k, v = (torch.randn(n * seqs, heads, hd, device="cuda", generator=gen) for _ in range(2))
    c.append(0, k, v, seqs=at, positions=pos)
    k, v = (x.double().view(seqs, n, heads, hd) for x in c.read(0, at, pos))
    q = 4 * torch.randn(seqs, heads, hd, device="cuda", generator=gen)
    got = c.attention(0, q).double()
    c.sync_status()
    w = torch.softmax(torch.einsum("shd,snhd->shn", q.double(), k) / hd ** 0.5, -1)
    want = torch.einsum("shn,snhd->shd", w, v)
    assert ((got - want).norm() / want.norm()).item() <= 5.5e-7


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_offsets_past_32_bits(fmt):
    """Pages whose bytes begin past 2^32, in the second layer too."""
    nkv, hd, R = 32, 128, 64
    pb = ref.Pages(fmt, nkv, hd, R).page_bytes
    n_pages = (1 << 32) // pb + 40
    c = kv.KVCache(n_layers=2, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=n_pages, n_seqs=2, max_pages=4)
    c.pool.fill_(0xFF)
    c.table[0, :3] = ints([n_pages - 1, 0, n_pages - 2])
    c.lens[0] = 150
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(150, nkv, hd, device="cuda", generator=gen) for _ in range(2))
    seqs, pos = ints([0] * 150), ints(range(150))
    c.append(1, k, v, seqs=seqs, positions=pos)
    kk, vv = c.read(1, seqs, pos)
    q = torch.randn(1, nkv, hd, device="cuda", generator=gen)
    out = c.attention(1, q, seqs=ints([0]))
    c.sync_status()
    kd, vd = kk.double(), vv.double()
    if fmt == "bf16":
        assert torch.equal(kk, k.bfloat16().float()) and torch.equal(vv, v.bfloat16().float())
    w = torch.softmax(torch.einsum("hd,nhd->hn", q[0].double(), kd) / hd ** 0.5, -1)
    o = torch.einsum("hn,nhd->hd", w, vd)
    assert (out[0].double() - o).abs().max() < 2e-5     # values of order one, 150 rows


def test_attention_in_graphs_and_streams():
    """Captured with lengths that change between replays, two graphs with a workspace each, another stream."""
    f = Filled("bf16", 2, 64, 16, [100, 260], seed=6)
    q = torch.randn(2, 4, 64, device="cuda")
    out_a, out_b = torch.empty_like(q), torch.empty_like(q)
    ws_a, ws_b = f.cache.workspace(), f.cache.workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f.cache.attention(f.layer, q, out=out_a, workspace=ws_a)
    torch.cuda.current_stream().wait_stream(side)
    f.check(q, out_a, range(2))
    graphs = []
    for out, ws, win in ((out_a, ws_a, 0), (out_b, ws_b, 40)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f.cache.attention(f.layer, q, out=out, workspace=ws, window=win, sinks=2 if win else 0)
        graphs.append(g)
    k, v = f.k, f.v
    for lens in ([100, 260], [3, 0], [99, 17]):
        f.cache.lens.copy_(ints(lens))
        q.copy_(torch.randn_like(q))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        f.cache.sync_status()
        for out, win in ((out_a, 0), (out_b, 40)):
            rows = [ref.visible(n, win, 2 if win else 0) for n in lens]
            f.k, f.v = [a[:, r] for a, r in zip(k, rows)], [a[:, r] for a, r in zip(v, rows)]
            f.check(q, out, range(2), what=f"window {win}, lengths {lens}")
    with pytest.raises(ValueError, match="workspace"):
        f.cache.attention(f.layer, q, stream=side)


def test_results_made_for_a_stream_are_made_on_it():
    """A call on a stream of its own while the current one is busy: nothing queued there may touch its results."""
    f = Filled("q4", 2, 64, 16, [100, 260], seed=9)
    q = torch.randn(2, 4, 64, device="cuda")
    seqs, pos, ws = ints([1, -1, 0]), ints([259, 0, 99]), f.cache.workspace()
    want = f.cache.read(f.layer, seqs, pos)
    outs = f.cache.attention(f.layer, q), f.cache.attention(f.layer, q, seqs=ints([0, -1]))
    some = ints([0, -1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)   # about 10 ms
        got = f.cache.read(f.layer, seqs, pos, stream=stream)
        got_outs = (f.cache.attention(f.layer, q, workspace=ws, stream=stream),
                    f.cache.attention(f.layer, q, seqs=some, workspace=ws, stream=stream))
        torch.cuda.synchronize()
        for a, b in zip(got + got_outs, want + outs):
            assert torch.equal(a, b)


def test_calls_from_another_device(monkeypatch):
    """Another device is current: calls go to the cache's, and a capture is noticed there (a graph's own
    workspace is never kept for other calls)."""
    f = Filled("bf16", 2, 64, 16, [100, 2600], seed=10)
    q = torch.randn(2, 4, 64, device="cuda")
    want = f.cache.attention(f.layer, q)
    g, out, kept, inside = torch.cuda.CUDAGraph(), torch.empty_like(q), dict(f.cache._workspaces), []
    here = kv._capturing

    class Entered(torch.cuda.device):
        def __enter__(self):
            inside.append(1)
            return super().__enter__()

        def __exit__(self, *error):
            inside.pop()
            return super().__exit__(*error)

    with torch.cuda.graph(g):
        monkeypatch.setattr(torch.cuda, "device", Entered)
        monkeypatch.setattr(kv, "_current_device", lambda: f.cache.device.index + (not inside))
        monkeypatch.setattr(kv, "_capturing", lambda: bool(inside) and here())  # (the other device captures nothing)
        f.cache.attention(f.layer, q, out=out)
        monkeypatch.undo()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and f.cache._workspaces == kept


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_without_workspaces_on_streams_and_in_graphs(fmt):
    """Calls that share nothing but the cache: two streams at once, and two graphs replayed beside them."""
    f = Filled(fmt, 2, 128, 16, [3000, 2500], seed=8)
    qs = [torch.randn(2, 4, 128, device="cuda") for _ in range(4)]
    want = [f.cache.attention(f.layer, q).clone() for q in qs]
    f.check(qs[0], want[0], range(2))
    outs = [torch.empty_like(q) for q in qs]
    graphs = []
    for i in (2, 3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f.cache.attention(f.layer, qs[i], out=outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(20):
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i < 2:
                    f.cache.attention(f.layer, qs[i], out=outs[i])
                else:
                    graphs[i - 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    f.cache.sync_status()


# ---- rows ------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nkv,hd,R", [(1, 64, 16), (3, 128, 48), (8, 64, 128), (5, 128, 16)])
def test_append_writes_the_documented_bytes(fmt, io, nkv, hd, R):
    rng = np.random.default_rng(nkv + hd)
    p = ref.Pages(fmt, nkv, hd, R)
    n_pages, n_seqs = 9, 4
    pool = rng.integers(0, 256, (2, n_pages, p.page_bytes)).astype(np.uint8)
    table = np.array([[8, 1], [3, 2], [0, 7], [-1, -1]], np.int32)
    c = kv.KVCache(n_layers=2, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, pool=torch.from_numpy(pool).cuda(),
                   table=ints(table), lens=ints([R + 1, R, 2 * R, 0]), refs=ints(np.ones(n_pages)))
    seqs = [0, 2, -1, 1, 0, 2, 0]
    pos = [0, 2 * R - 1, 5, R - 1, R, 3, 7]
    n = len(seqs)
    x = torch.randn(2, n, nkv, hd, device="cuda")
    x[0, 0] *= 300
    x[1, 1] = 0                                   # a block of zeros
    x[0, 3, 0, :32] *= 1e-6                       # a scale below fp16's normal numbers
    x[1, 3, 0, :32] = 1e-9                        # one that rounds to zero
    x = x.to(io)
    wide = torch.zeros(n, nkv + 2, hd, device="cuda", dtype=io)  # rows wider than what is taken
    wide_v = torch.zeros_like(wide)
    wide[:, 1:nkv + 1], wide_v[:, 1:nkv + 1] = x[0], x[1]
    k, v = wide[:, 1:nkv + 1], wide_v[:, 1:nkv + 1]
    c.append(1, k, v, seqs=ints(seqs), positions=ints(pos))
    want = pool.copy()
    for t, (s, at) in enumerate(zip(seqs, pos)):
        if s >= 0:
            for which, src in ((0, f32(k)), (1, f32(v))):
                for h in range(nkv):
                    p.put(want[1, table[s, at // R]], which, h, at % R, src[t, h])
    got = c.pool.cpu().numpy()
    assert np.array_equal(got, want)              # nothing else changed either
    c.sync_status()
    # and back, in both types
    for dt in (torch.float32, torch.bfloat16):
        bk = torch.full((n, nkv, hd), 9.0, device="cuda", dtype=dt)
        bv = bk.clone()
        c.read(1, ints(seqs), ints(pos), k_out=bk, v_out=bv)
        for t, (s, at) in enumerate(zip(seqs, pos)):
            for which, b in ((0, bk), (1, bv)):
                if s < 0:
                    assert torch.all(b[t] == 9)
                    continue
                val = p.values(want[1, table[s, at // R]])[which, :, at % R].astype(np.float32)
                val = ref.bf16_value(ref.bf16_bits(val)) if dt == torch.bfloat16 else val
                assert np.array_equal(f32(b[t]), val)
    c.sync_status()
    # last rows, without lists
    c.lens.copy_(ints([R + 1, R, 2 * R, 1]))
    c.table[3, 0] = 4
    c.append(0, k[:4], v[:4])
    kk, _ = c.read(0, ints(range(4)))
    k2, _ = c.read(0, ints(range(4)), ints([R, R - 1, 2 * R - 1, 0]))
    assert torch.equal(kk, k2)
    c.sync_status()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 700])
def test_rows_at_other_alignments(fmt, io, rows):
    """Rows that begin 16 bytes past a multiple of 32, or are an odd number of 16 bytes apart."""
    nkv, hd, R = 8, 64, 16
    c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=-(-rows // R), n_seqs=1,
                   max_pages=-(-rows // R))
    c.extend(None, ints([rows]))
    seqs, pos, step = ints([0] * rows), ints(range(rows)), 16 // (4 if io == torch.float32 else 2)

    def placed(offset, gap):
        width = nkv * hd + gap
        flat = torch.full((offset + rows * width,), 7.0, dtype=io, device="cuda")
        return flat, flat[offset:].view(rows, width)[:, :nkv * hd].view(rows, nkv, hd)

    k, v = (torch.randn(rows, nkv, hd, device="cuda").to(io) for _ in range(2))
    want = None
    for offset, gap in ((0, 0), (step, 0), (0, step), (step, step), (0, 2 * step)):
        (_, kin), (_, vin) = placed(offset, gap), placed(offset, gap)
        kin.copy_(k)
        vin.copy_(v)
        c.pool.fill_(0xFF)
        c.append(0, kin, vin, seqs=seqs, positions=pos)
        (kf, ko), (vf, vo) = placed(offset, gap), placed(offset, gap)
        c.read(0, seqs, pos, k_out=ko, v_out=vo)
        c.sync_status()
        want = want or (c.pool.clone(), ko.clone(), vo.clone())
        assert torch.equal(c.pool, want[0]) and torch.equal(ko, want[1]) and torch.equal(vo, want[2]), (offset, gap)
        for flat, rest in ((kf, ko), (vf, vo)):   # what lies between the rows stays
            rest.fill_(7.0)
            assert (flat == 7.0).all(), (offset, gap)
    if fmt == "bf16":
        assert torch.equal(want[1], k.bfloat16().to(io))


def test_append_ties_and_extremes():
    """Quotients on and next to a half, at 24 bits; blocks with NaN or infinity; values past fp16's range."""
    hd, R = 64, 16
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=hd, page_rows=R, fmt="q4", n_pages=8, n_seqs=1, max_pages=8)
    c.extend(n_new=ints([128]))
    rng = np.random.default_rng(8)
    x = np.zeros((128, 2, 32), np.float32)
    for t in range(100):
        for b in range(2):
            s = np.float16(rng.uniform(0.01, 3) * 2.0 ** rng.integers(-14, 10))
            x[t, b, 0] = np.float32(s) * 7        # the block's largest magnitude gives this scale
            half = (rng.integers(-7, 7, 31) + 0.5).astype(np.float64) * np.float64(s)
            y = half.astype(np.float32)
            x[t, b, 1:] = np.where(rng.random(31) < 0.4, y, np.nextafter(y, np.float32(rng.choice([-9e9, 9e9]))))
    x[100:104] = rng.normal(0, 1, (4, 2, 32))
    x[100, 0, 3], x[101, 1, 31], x[102, 0, 0] = np.nan, np.inf, -np.inf
    x[104, 0, 5], x[104, 0, 6], x[104, 1, 7] = 3e38, -2e5, 4.6e5
    x[105, 0, 0], x[105, 1, 0] = 1e-45, 5e-7
    x[106, 0, :2] = [65504 * 7, 65519 * 7]
    k = torch.from_numpy(x.reshape(128, 1, hd)).cuda()
    c.append(0, k, -k, seqs=ints([0] * 128), positions=ints(range(128)))
    c.sync_status()
    p = ref.Pages("q4", 1, hd, R)
    pool, table = c.pool.cpu().numpy()[0], c.table.cpu().numpy()[0]
    want = np.zeros_like(pool)
    for t in range(128):
        p.put(want[table[t // R]], 0, 0, t % R, x[t].ravel())
        p.put(want[table[t // R]], 1, 0, t % R, -x[t].ravel())
    got_v, want_v = (np.stack([p.values(a[q]) for q in table]) for a in (pool, want))
    assert np.array_equal(np.isnan(got_v), np.isnan(want_v)) and np.isnan(got_v).any()
    ok = ~np.isnan(want_v)
    assert np.array_equal(got_v[ok], want_v[ok])


def test_rows_out_of_range_are_skipped():
    c = kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, page_rows=16, n_pages=4, n_seqs=2, max_pages=2)
    c.extend(n_new=ints([20, 3]))
    c.pool.fill_(3)
    before = c.pool.clone()
    x = torch.randn(6, 2, 64, device="cuda")
    c.append(0, x, x, seqs=ints([2, 0, 0, 1, 1, 70000]), positions=ints([0, -1, 32, 16, 1 << 30, 0]))
    with pytest.raises(dec.DecError) as e:
        c.sync_status()
    assert e.value.code == dec.DEC_ERR_DEVICE
    assert torch.equal(c.pool, before)
    keep = torch.full((2, 2, 64), 4.0, device="cuda")
    c.read(0, ints([5, 1]), ints([0, 40]), k_out=keep, v_out=keep.clone())
    with pytest.raises(dec.DecError):
        c.sync_status()
    assert torch.all(keep == 4)
    c.release(ints([1]))
    c.append(0, x[:2], x[:2])                         # sequence 1 has no last row
    with pytest.raises(dec.DecError):
        c.sync_status()


# ---- pages ------------------------------------------------------------------------

def _same(c, m, pool):
    assert np.array_equal(c.table.cpu().numpy(), m.table)
    assert np.array_equal(c.lens.cpu().numpy(), m.lens)
    assert np.array_equal(c.refs.cpu().numpy(), m.refs)
    assert np.array_equal(c.pool.cpu().numpy(), pool)


@pytest.mark.parametrize("n_pages,n_seqs,max_pages,R,fmt", [
    (40, 10, 12, 16, "bf16"), (7, 3, 5, 32, "q4"), (2500, 70, 64, 16, "q4"), (1, 1, 1, 16, "bf16"), (1500, 1300, 3, 16, "q4")])
def test_pages_follow_the_model(n_pages, n_seqs, max_pages, R, fmt):
    """A random walk of all page calls, errors among them, state by state and page by page."""
    rng = np.random.default_rng(n_pages)
    c = kv.KVCache(n_layers=2, n_kv_heads=1, head_dim=64, page_rows=R, fmt=fmt, n_pages=n_pages, n_seqs=n_seqs,
                   max_pages=max_pages)
    pool = rng.integers(0, 256, tuple(c.pool.shape)).astype(np.uint8)
    c.pool.copy_(torch.from_numpy(pool))
    m = ref.Model(n_pages, n_seqs, max_pages, R)
    seen = 0
    for step in range(60):
        op, k = rng.integers(0, 6), min(n_seqs, int(rng.integers(1, n_seqs + 1)))
        some = rng.permutation(n_seqs)[:k]
        m.copies = []
        if op == 0:
            add = rng.integers(0, 2 * R, k)
            if rng.random() < 0.2:
                add[0] = rng.choice([-1, 10 ** 9])
            if rng.random() < 0.2:
                some[-1] = some[0]
            if rng.random() < 0.3:
                some[0] = -1
            m.extend(some, add)
            c.extend(ints(some), ints(add))
        elif op == 1:
            m.extend(range(n_seqs))
            c.extend()
        elif op == 2:
            kids = [s for s in some if m.lens[s] == 0] if rng.random() < 0.8 else list(some)
            parents = [int(rng.choice(np.setdiff1d(np.arange(n_seqs), kids))) if len(kids) < n_seqs else 0 for _ in kids]
            if kids:
                if rng.random() < 0.2:
                    parents[0] = int(rng.choice([-1, n_seqs, kids[-1]]))
                m.fork(parents, kids)
                c.fork(ints(parents), ints(kids))
        elif op == 3:
            some = np.concatenate((some[:1], some))[:n_seqs]
            m.release(some)
            c.release(ints(some))
        elif op == 4:
            w, s = int(rng.integers(1, 3 * R)), int(rng.integers(0, 2 * R))
            m.release(range(n_seqs), w, s)
            c.release(window=w, sinks=s)
        else:
            m.compact()
            c.compact()
        for a, b in m.copies:
            pool[:, b] = pool[:, a]
        _same(c, m, pool)
        if m.bits:
            seen += 1
            with pytest.raises(dec.DecError):
                c.sync_status()
            m.bits = 0
        c.sync_status()
    assert seen or n_pages > 2000


def test_page_calls_refuse_without_change():
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, n_pages=6, n_seqs=4, max_pages=4)
    c.extend(ints([0, 1]), ints([40, 20]))
    c.sync_status()
    state = [t.clone() for t in (c.table, c.lens, c.refs)]
    calls = [
        (lambda: c.extend(ints([2, 2])), "bad list"),
        (lambda: c.extend(ints([2, 4])), "index"),
        (lambda: c.extend(ints([2, 3]), ints([1, -1])), "index"),
        (lambda: c.extend(ints([2, 3]), ints([16, 1])), "no free pages"),
        (lambda: c.extend(ints([2]), ints([65])), "no free pages"),
        (lambda: c.fork(ints([0]), ints([1])), "bad list"),          # not empty
        (lambda: c.fork(ints([0, 1]), ints([2, 2])), "bad list"),
        (lambda: c.fork(ints([0, 2]), ints([2, 3])), "bad list"),    # a child that is a parent
        (lambda: c.fork(ints([0]), ints([4])), "index"),
        (lambda: c.fork(ints([0, 1]), ints([2, 3])), "no free pages"),
    ]
    for call, text in calls:
        call()
        with pytest.raises(dec.DecError, match=text):
            c.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(state, (c.table, c.lens, c.refs)))
    with pytest.raises(dec.DecError):
        c.extend(ints([0, 1, 2, 3, 0]))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_a_run_of_all_calls(fmt):
    """Prefill, decode with a window, fork, release, compact and decode on, against rows kept on the host:
    every sequence's attention at every step, the calls captured in one graph per step."""
    nkv, group, hd, R, W, S = 2, 3, 64, 16, 60, 4
    n_seqs = 6
    c = kv.KVCache(n_layers=2, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=60, n_seqs=n_seqs, max_pages=12)
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows = [[np.zeros((2, nkv, 0, hd)) for _ in range(n_seqs)] for _ in range(2)]   # [layer][seq]

    def stored(x):
        x = f32(x)
        if fmt == "bf16":
            return ref.bf16_value(ref.bf16_bits(x)).astype(np.float64)
        return ref.q4_value(*ref.q4_encode(x))

    def note(layer, seqs, k, v):
        both = np.stack((stored(k), stored(v)))                                     # [2][n][head][d]
        for t, s in enumerate(seqs):
            rows[layer][s] = np.concatenate((rows[layer][s], both[:, t][:, :, None]), 2)

    first = {0: 70, 1: 33, 3: 1}
    c.extend(ints(list(first)), ints(list(first.values())))
    seqs = [s for s, n in first.items() for _ in range(n)]
    pos = [j for n in first.values() for j in range(n)]
    for layer in range(2):
        k, v = (torch.randn(len(seqs), nkv, hd, device="cuda", generator=gen) for _ in range(2))
        c.append(layer, k, v, seqs=ints(seqs), positions=ints(pos))
        note(layer, seqs, k, v)
    live = [0, 1, 3]
    k = torch.zeros(2, n_seqs, nkv, hd, device="cuda")
    v = torch.zeros_like(k)
    q = torch.zeros(2, n_seqs, nkv * group, hd, device="cuda")
    out = torch.zeros_like(q)
    lst = ints([-1] * n_seqs)
    ws = c.workspace()
    graph = torch.cuda.CUDAGraph()

    def step():
        c.extend(lst)
        for layer in range(2):
            c.append(layer, k[layer], v[layer], seqs=lst)
            c.attention(layer, q[layer], seqs=lst, window=W, sinks=S, out=out[layer], workspace=ws)
        c.release(lst, window=W, sinks=S)

    with torch.cuda.graph(graph):
        step()
    for t in range(30):
        if t == 6:
            c.fork(ints([0, 0, 3]), ints([2, 4, 5]))
            for layer in range(2):
                for a, b in ((0, 2), (0, 4), (3, 5)):
                    rows[layer][b] = rows[layer][a].copy()
            live = [0, 1, 2, 3, 4, 5]
        if t == 15:
            c.release(ints([0, 1]))
            for layer in range(2):
                rows[layer][0] = rows[layer][1] = np.zeros((2, nkv, 0, hd))
            live = [5, 3, 2, 4]
        if t in (16, 23):
            c.compact()
            named = c.table[c.table >= 0].unique()
            assert int(named.max()) == len(named) - 1
        lst.copy_(ints(live + [-1] * (n_seqs - len(live))))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        graph.replay()
        c.sync_status()
        for layer in range(2):
            note(layer, live, k[layer, :len(live)], v[layer, :len(live)])
            for i, s in enumerate(live):
                a = rows[layer][s]
                vis = ref.visible(a.shape[2], W, S)
                o, size, dots = ref.attention(f32(q[layer, i]).astype(np.float64), a[0][:, vis], a[1][:, vis], hd ** -0.5)
                tol = size * (2 * (hd + 8) * 2.0 ** -24 * dots[:, None] + 2.0 ** -16) + 1e-30   # 64 rows: n 2^-23 < 2^-17
                assert np.all(np.abs(f32(out[layer, i]) - o) <= tol), (t, layer, s)
    refs = np.bincount(c.table.cpu().numpy()[c.table.cpu().numpy() >= 0], minlength=60)
    assert np.array_equal(refs, c.refs.cpu().numpy())


def test_python_checks_tensors():
    c = kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, n_pages=2, n_seqs=2, max_pages=1)
    x = torch.zeros(2, 2, 64, device="cuda")
    bad = [
        lambda: c.append(0, x.half(), x.half()), lambda: c.append(0, x, x.bfloat16()), lambda: c.append(0, x, x[:1]),
        lambda: c.append(0, x[:, :1], x[:, :1]), lambda: c.append(0, x.cpu(), x.cpu()),
        lambda: c.append(0, x, x, seqs=ints([0])), lambda: c.append(0, x, x, seqs=ints([0, 1]).long()),
        lambda: c.append(0, x.transpose(0, 1), x.transpose(0, 1).contiguous()),
        lambda: c.read(0, ints([0]), k_out=x), lambda: c.attention(0, x, out=x[:1]),
        lambda: c.attention(0, x, out=x.bfloat16()), lambda: c.extend(ints([0]), ints([1, 2])),
        lambda: c.fork(ints([0]), ints([1, 1])), lambda: c.extend(torch.zeros(1, dtype=torch.int32)),
        lambda: kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, pool=c.pool, table=c.table, lens=c.lens[:1], refs=c.refs),
        lambda: kv.KVCache(n_layers=2, n_kv_heads=2, head_dim=64, pool=c.pool, table=c.table, lens=c.lens, refs=c.refs),
        lambda: kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, pool=c.pool.cpu(), table=c.table.cpu(),
                           lens=c.lens.cpu(), refs=c.refs.cpu()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(dec.DecError):
        c.attention(0, torch.zeros(2, 3, 64, device="cuda"))     # 3 heads over 2
    with pytest.raises(dec.DecError):
        c.attention(5, x)
    c.sync_status()
