"""8-bit pages and rotary positions on the GPU against their 64-bit statements.

Tolerances of attention.  As over the other pages (tests/test_gpu_kv_cache.py): a
score is off by at most (d + 8) * 2^-24 of sum |q||k| scale (the roundings of its sum
and the split of q among them), a weight is an exponential good to 2^-20, n weights
are summed and n products accumulated in fp32, so an output is off by at most
sum_j w_j |v_j| * (2 * ds + 2 * n * 2^-24 + 2^-19), plus half a step of its own type.
The codes and the scales are exact, so over 8-bit pages only the weights are cut: fp32
results take them in two fp16 pieces (2^-22 of a weight), bf16 results as one (2^-11),
and both are off by at most 2^-34 more where the largest weight counts 1 or more: 2^-24 is
fp16's least step, of which half is lost, and the weights enter times 2^9, 2^-25 / 2^9.
Writing and reading are exact, and so compared bit for bit.
"""
import numpy as np
import pytest

import kv8_reference as ref
import kv_reference as ref4
from transformer_layer_decode_gb300 import dec, kv, rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


class Filled:
    """A cache of 8 bits whose sequences have the given lengths, its pool random bytes (scales of NaN among
    them) but for the blocks that a query sees, which have powers of two as scales."""

    def __init__(self, nkv, hd, R, lens, *, layers=2, layer=1, seed=0, window=0, sinks=0, spare=3, room=1,
                 exponents=(-8, 1), codes=None):
        rng = np.random.default_rng(seed)
        self.pages, self.lens, self.layer, self.R = ref.Pages8(nkv, hd, R), list(lens), layer, R
        width = max(-(-room // R), max(-(-n // R) for n in lens))
        table = np.full((len(lens), width), -1, np.int32)
        seen = [ref4.visible(n, window, sinks) for n in lens]
        wanted = [(s, i) for s, v in enumerate(seen) for i in np.unique(v // R)]
        order = rng.permutation(len(wanted) + spare)
        for (s, i), p in zip(wanted, order):
            table[s, i] = p
        pool = rng.integers(0, 256, (layers, len(order), self.pages.page_bytes)).astype(np.uint8)
        self.k, self.v = [], []
        for s, v in enumerate(seen):
            for i in np.unique(v // R):
                page = pool[layer, table[s, i]]
                c, sc = self.pages.parts(page)
                for one in sc:
                    one[:] = np.nan
                for b in np.unique(v[v // R == i] % R // 16):
                    for half in range(2):
                        sc[half][:, b] = 2.0 ** rng.integers(*exponents, nkv)
                if codes:
                    for half in c:
                        half[:] = codes(rng, half.shape)
            both = np.stack([self.pages.values(pool[layer, p]) for p in table[s, np.unique(v // R)]]) if len(v) else None
            at = np.searchsorted(np.unique(v // R), v // R)
            kv_rows = both[at, :, :, v % R] if len(v) else np.zeros((0, 2, nkv, hd))
            self.k.append(kv_rows[:, 0].transpose(1, 0, 2))
            self.v.append(kv_rows[:, 1].transpose(1, 0, 2))
        refs = np.bincount(table[table >= 0], minlength=len(order))
        self.pool = pool
        self.cache = kv.KVCache(n_layers=layers, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt="q8",
                                pool=torch.from_numpy(pool).cuda(), table=ints(table), lens=ints(lens), refs=ints(refs))

    def check(self, q, got, seqs, scale=None, what=""):
        scale = self.pages.d ** -0.5 if scale is None else scale
        bf16 = got.dtype == torch.bfloat16
        q, got = f64(q), f64(got)
        assert np.isfinite(got).all(), what
        for r, s in enumerate(seqs):
            if s < 0:
                continue
            o, size, dots = ref4.attention(q[r], self.k[s], self.v[s], scale)
            n = self.k[s].shape[1]
            ds = (self.pages.d + 8) * 2.0 ** -24 * np.abs(dots)[:, None]
            tol = size * (2 * ds + 2 * n * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** (-11 if bf16 else -22))
            if n:
                tol = tol + n * 2.0 ** -34 * np.abs(self.v[s]).max()
            tol = tol + (np.abs(o) + tol) * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-37
            bad = np.abs(got[r] - o) > tol
            assert not bad.any(), (what, r, s, n, np.argwhere(bad)[:4].tolist(), np.abs(got[r] - o)[bad][:4], tol[bad][:4])


# ---- rows ----------------------------------------------------------------------


def test_rows_of_one_block():
    """The smallest call: one row, then the next, then a larger one, which the others' codes follow."""
    p = ref.Pages8(1, 64, 16)
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, fmt="q8", n_pages=1, n_seqs=1, max_pages=1)
    c.pool.fill_(0xFF)                                    # NaN as scale
    page = c.pool.cpu().numpy()[0, 0].copy()
    rng = np.random.default_rng(0)
    for r, size in enumerate((1.0, 0.5, 40.0, 1e-3, 1e6)):
        x = (rng.normal(0, 1, (2, 1, 1, 64)) * size).astype(np.float32)
        c.extend()
        c.append(0, torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda())
        p.write(page, 0, {r: x[:, 0]})
        c.sync_status()
        codes, scales = p.parts(page)
        got_codes, got_scales = p.parts(c.pool.cpu().numpy()[0, 0])
        for i in range(2):
            assert got_scales[i][0, 0] == scales[i][0, 0] and np.array_equal(got_codes[i][0, :r + 1], codes[i][0, :r + 1])
    k, v = c.read(0, ints([0] * 5), ints(range(5)))
    assert np.array_equal(f64(k)[:, 0], p.values(page)[0, 0, :5]) and np.array_equal(f64(v)[:, 0], p.values(page)[1, 0, :5])


class Walk:
    """A cache and, beside it, its bytes as the statement makes them, call by call."""

    def __init__(self, nkv, hd, R, n_seqs, pages_each, *, layers=2, layer=1, seed=0):
        self.rng = np.random.default_rng(seed)
        self.p, self.layer, self.R = ref.Pages8(nkv, hd, R), layer, R
        n_pages = n_seqs * pages_each + 2
        self.pool = self.rng.integers(0, 256, (layers, n_pages, self.p.page_bytes)).astype(np.uint8)
        self.table = self.rng.permutation(n_pages)[:n_seqs * pages_each].reshape(n_seqs, pages_each).astype(np.int32)
        self.lens = np.zeros(n_seqs, np.int32)
        refs = np.bincount(self.table.ravel(), minlength=n_pages)
        self.cache = kv.KVCache(n_layers=layers, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt="q8",
                                pool=torch.from_numpy(self.pool.copy()).cuda(), table=ints(self.table),
                                lens=ints(self.lens), refs=ints(refs))
        self.live = {}                                    # (sequence, block): rows that hold something

    def rows(self, n, io, size):
        x = self.rng.normal(0, 1, (2, n, self.p.h, self.p.d)) * size
        t = torch.from_numpy(x.astype(np.float32)).cuda().to(io)
        return t, t.float().cpu().numpy()

    def append(self, plan, io, size, *, positions=True, mode="append"):
        """plan: [(sequence or -1, position)]"""
        t, x = self.rows(len(plan), io, size)
        if positions:
            self.cache.append(self.layer, t[0], t[1], seqs=ints([s for s, _ in plan]), positions=ints([p for _, p in plan]))
        else:
            self.cache.append(self.layer, t[0], t[1], seqs=ints([s for s, _ in plan]))
        self.note(plan, x)

    def note(self, plan, x):
        by_block = {}
        for i, (s, pos) in enumerate(plan):
            if s >= 0:
                by_block.setdefault((s, pos // 16), {})[pos % 16] = x[:, i]
        for (s, b), rows in by_block.items():
            page = self.pool[self.layer, self.table[s, b * 16 // self.R]]
            self.p.write(page, b * 16 % self.R // 16, rows)
            first = min(rows)
            self.live[s, b] = {r for r in self.live.get((s, b), set()) if r < first} | set(rows)

    def check(self, io=torch.float32):
        self.cache.sync_status()
        got = self.cache.pool.cpu().numpy()
        for (s, b), rows in self.live.items():
            page, block = self.table[s, b * 16 // self.R], b * 16 % self.R // 16
            (ck, cv), (sk, sv) = self.p.parts(self.pool[self.layer, page])
            (gk, gv), (hk, hv) = self.p.parts(got[self.layer, page])
            at = 16 * block + np.array(sorted(rows))
            for want, have, scale, h in ((ck, gk, sk, hk), (cv, gv, sv, hv)):
                assert np.array_equal(scale[:, block], h[:, block], equal_nan=True), (s, b, scale[:, block], h[:, block])
                fine = np.isfinite(scale[:, block])
                assert np.array_equal(want[fine][:, at], have[fine][:, at]), (s, b)
        untouched = [i for i in range(got.shape[0]) if i != self.layer]
        assert np.array_equal(got[untouched], self.pool[untouched])
        plan = [(s, 16 * b + r) for (s, b), rows in self.live.items() for r in rows]
        k, v = self.cache.read(self.layer, ints([s for s, _ in plan]), ints([p for _, p in plan]), dtype=io)
        for i, x in enumerate((k, v)):
            want = np.stack([self.p.values(self.pool[self.layer, self.table[s, p // self.R]])[i, :, p % self.R]
                             for s, p in plan])
            want = torch.from_numpy(want).to(io).double().numpy()
            assert np.array_equal(f64(x), want, equal_nan=True)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nkv,hd,R", [(2, 64, 128), (1, 128, 16), (3, 128, 48), (5, 64, 16), (8, 128, 64)])
def test_append_and_read(io, nkv, hd, R):
    """A decode step by step over ragged sequences, rows that grow and shrink in size; then prompts in pieces."""
    w = Walk(nkv, hd, R, 6, -(-160 // R), seed=nkv + hd + R)
    w.append([(0, i) for i in range(37)] + [(2, i) for i in range(5)], io, 1.0)
    w.check(io)
    lens = np.array([37, 0, 5, 0, 0, 0])
    for step in range(20):
        lens = lens + 1
        w.cache.lens.copy_(ints(lens))
        w.append([(s, int(n) - 1) for s, n in enumerate(lens)], io, 2.0 ** w.rng.integers(-3, 4), positions=False)
    w.check(io)
    for s in (4, 1, 5):                                   # what comes behind position 20 of a sequence, in pieces
        at = 20
        for n in (3, 1, 30, 16, 2):
            w.append([(s, at + i) for i in range(n)], io, 2.0 ** w.rng.integers(-2, 3))
            at += n
    w.check(io)
    w.append([(1, 10), (1, 11), (2, 0), (4, 33)], io, 1.0)  # back over rows that were there
    w.check(io)


@pytest.mark.parametrize("n", [1, 2, 40, 511, 512, 513, 1500])
@pytest.mark.parametrize("order", ["runs", "across", "shuffled"])
def test_lists_in_any_order(n, order):
    """Short lists and long ones (which are looked through in another way), rows of a block together or apart,
    padding among them."""
    w = Walk(2, 64, 64, 8, -(-(n // 8 + 70) // 64), seed=n)
    for turn in range(3):
        starts = w.rng.integers(0, 60, 8)
        plan = [(s, int(starts[s]) + i) for s in range(8) for i in range(-(-n // 8))][:n]
        if order == "across":
            plan.sort(key=lambda x: (x[1], x[0]))
        if order == "shuffled":
            w.rng.shuffle(plan)
            plan = [tuple(int(v) for v in x) for x in plan]
        if n > 10:
            plan[n // 3] = (-1, 7)
            plan[n - 1] = (-5, 0)
        for s, b in {(s, p // 16) for s, p in plan if s >= 0} - set(w.live):  # begun before, with some scale
            for part in w.p.parts(w.pool[w.layer, w.table[s, b * 16 // 64]])[1]:
                part[:, b * 16 % 64 // 16] = 2.0 ** -6
        w.cache.pool.copy_(torch.from_numpy(w.pool))
        w.append(plan, torch.float32, 2.0 ** (turn - 1))
        w.check()
        w.pool[:] = w.cache.pool.cpu().numpy()


@pytest.mark.parametrize("hd", [64, 128])
def test_values_at_the_ends(hd):
    """Zeros, subnormal and largest numbers, borders of a scale, ties; NaN and infinities make a block NaN until
    its first row is written again."""
    w = Walk(1, hd, 16, 10, 1, seed=hd)
    rows = np.zeros((10, 1, hd), np.float32)
    rows[1, 0, 3] = 1e-45
    rows[2, 0, :5] = [3e-38, -1e-39, 2e-38, 5e-41, 0]
    rows[3, 0, :4] = [3.4028235e38, -3.4028235e38, 1e38, 2.0 ** 121 * 0.5]
    rows[4, 0, :4] = [127.0, 0.5, 1.5, -2.5]
    rows[5, 0, :4] = [np.nextafter(np.float32(127), np.float32(128)), 1.0, 3.0, -5.0]
    rows[6, 0, :3] = [127.0 * 2.0 ** 121, -127.0 * 2.0 ** 121, 2.0 ** 120]
    rows[7, 0, 1] = np.nan
    rows[8, 0, hd - 1] = -np.inf
    rows[9, 0] = np.arange(hd) - 63.5
    x = np.stack([rows, rows[::-1]])
    t = torch.from_numpy(x.copy()).cuda()
    plan = [(s, 0) for s in range(10)]
    w.cache.append(1, t[0], t[1], seqs=ints(range(10)), positions=ints([0] * 10))
    w.note(plan, x)
    w.check()
    assert np.isnan(f64(w.cache.read(1, ints([7, 8]), ints([0, 0]))[0])).all()
    w.append([(s, 1) for s in range(10)], torch.float32, 1.0)   # stays NaN
    w.check()
    assert np.isnan(f64(w.cache.read(1, ints([7, 8]), ints([1, 1]))[0])).all()
    w.append([(s, 0) for s in range(10)], torch.float32, 1.0)   # begun again
    w.check()
    assert np.isfinite(f64(w.cache.read(1, ints(range(10)), ints([0] * 10))[0])).all()


def test_bad_rows_are_skipped():
    w = Walk(2, 64, 16, 4, 2, seed=1)
    before = w.cache.pool.clone()
    w.cache.table[2, 1] = -1
    w.cache.table[3, 0] = 99
    k = torch.ones(7, 2, 64, device="cuda")
    for seqs, positions in (([4, 0, 2, 3, 0, -1, 70000], [0, 32, 16, 3, -1, 0, 1]),):
        w.cache.append(1, k, k, seqs=ints(seqs), positions=ints(positions))
        with pytest.raises(dec.DecError, match="index"):
            w.cache.sync_status()
        out = torch.full((7, 2, 64), 5.0, device="cuda")
        w.cache.read(1, ints(seqs), ints(positions), k_out=out, v_out=out.clone())
        with pytest.raises(dec.DecError, match="index"):
            w.cache.sync_status()
        assert bool((out == 5).all())
    assert torch.equal(w.cache.pool, before)
    many = torch.ones(600, 2, 64, device="cuda")             # the long list's way
    w.cache.append(1, many, many, seqs=ints([4, -1, 70000] * 200), positions=ints([0] * 600))
    with pytest.raises(dec.DecError, match="index"):
        w.cache.sync_status()
    assert torch.equal(w.cache.pool, before)


def test_appends_of_two_streams_share_nothing():
    """Calls on other layers, and on other blocks of a layer, may overlap."""
    w = Walk(2, 64, 64, 16, 12, layers=2, layer=1, seed=5)
    other = [(s, i) for s in range(8, 16) for i in range(100)]
    mine = [(s, i) for s in range(8) for i in range(100)]
    t, x = w.rows(800, torch.float32, 1.0)
    u, y = w.rows(800, torch.float32, 1.0)
    lists = [(ints([s for s, _ in p]), ints([i for _, i in p])) for p in (mine, other)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (seqs, pos), rows, layer, st in ((lists[0], t, 1, streams[0]), (lists[1], u, 1, streams[1]),
                                             (lists[0], u, 0, streams[2])):
            w.cache.append(layer, rows[0], rows[1], seqs=seqs, positions=pos, stream=st)
    torch.cuda.synchronize()
    w.note(mine, x)
    w.note(other, y)
    w.layer = 0
    live, w.live = w.live, {}
    w.note(mine, y)
    got = w.cache.pool.cpu().numpy()
    for layer, blocks in ((1, live), (0, w.live)):
        for (s, b), rows in blocks.items():
            page, block = w.table[s, b * 16 // 64], b * 16 % 64 // 16
            (ck, cv), (sk, sv) = w.p.parts(w.pool[layer, page])
            (gk, gv), (hk, hv) = w.p.parts(got[layer, page])
            at = 16 * block + np.array(sorted(rows))
            assert np.array_equal(sk[:, block], hk[:, block]) and np.array_equal(sv[:, block], hv[:, block])
            assert np.array_equal(ck[:, at], gk[:, at]) and np.array_equal(cv[:, at], gv[:, at])


# ---- attention -----------------------------------------------------------------

SHAPES = [  # kv heads, group, head_dim, page rows
    (2, 4, 64, 128), (1, 1, 128, 16), (3, 2, 128, 64), (2, 8, 128, 32), (1, 12, 64, 48), (4, 3, 64, 16), (2, 5, 128, 128),
]


@pytest.mark.parametrize("room", [1, 40000])  # rows that a table has room for: short ones are not cut between CTAs
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nkv,group,hd,R", SHAPES)
def test_attention_all_rows(io, nkv, group, hd, R, room):
    lens = [0, 1, 15, 16, 17, R, R + 1, 2 * R - 1, 333, 2]
    f = Filled(nkv, hd, R, lens, seed=nkv * 100 + hd + R, room=room)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(len(lens), nkv * group, hd, device="cuda", generator=g).to(io)
    out = f.cache.attention(f.layer, q)
    f.cache.sync_status()
    f.check(q, out, range(len(lens)))
    assert not out[0].any()


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (50, 1), (64, 70), (100, 33)])
@pytest.mark.parametrize("nkv,group,hd,R", [(2, 4, 64, 48), (2, 2, 128, 64)])
def test_attention_window(io, window, sinks, nkv, group, hd, R):
    """Rows that are not seen share a block with those that are, and hold any bytes; blocks that hold none have
    NaN for a scale."""
    lens = [0, 1, 17, 49, 100, 333, 700]
    f = Filled(nkv, hd, R, lens, seed=window + sinks, window=window, sinks=sinks)
    q = torch.randn(len(lens), nkv * group, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(io)
    out = f.cache.attention(f.layer, q, window=window, sinks=sinks)
    f.cache.sync_status()
    f.check(q, out, range(len(lens)))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("codes", ["ends", "small"])
def test_attention_codes_and_scales_far_apart(io, codes):
    """Codes at both ends, byte 0 among them; scales of blocks many powers of two apart, scores that do not decide."""
    make = (lambda rng, shape: rng.choice([0, 1, 255], shape)) if codes == "ends" else (lambda rng, shape: rng.integers(127, 130, shape))
    f = Filled(2, 128, 32, [5, 64, 500, 1000], seed=3, exponents=(-30, 4) if codes == "small" else (-12, -5), codes=make)
    q = 0.05 * torch.randn(4, 4, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(io)
    out = f.cache.attention(f.layer, q, scale=0.5)
    f.check(q, out, range(4), scale=0.5)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_attention_lists_strides_and_padding(io):
    lens = [40, 0, 129, 77]
    f = Filled(2, 64, 64, lens, seed=8)
    seqs = [2, -1, 0, 1, 3, 2, -7]
    wide = torch.randn(len(seqs), 10, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).to(io)
    q, out = wide[:, :6], torch.full((len(seqs), 9, 64), 3.0, device="cuda", dtype=io)
    f.cache.attention(f.layer, q, seqs=ints(seqs), out=out[:, 2:8])
    f.cache.sync_status()
    f.check(q, out[:, 2:8], seqs)
    assert bool((out[:, :2] == 3).all() and (out[:, 8:] == 3).all() and (out[1] == 3).all() and (out[6] == 3).all())


@pytest.mark.parametrize("n,lens", [(1, [30000]), (24, None), (200, None)])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_attention_cut_between_ctas(io, n, lens):
    """Long and ragged batches; the same call gives the same bits."""
    rng = np.random.default_rng(n)
    lens = lens or [int(x) for x in rng.integers(0, 3000 if n < 100 else 400, n)]
    f = Filled(2, 64, 128, lens, seed=n, layers=1, layer=0, exponents=(-7, -4))
    q = torch.randn(n, 8, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(io)
    out = f.cache.attention(0, q)
    f.check(q, out, range(n))
    assert torch.equal(out, f.cache.attention(0, q))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_attention_pages_that_are_none(io):
    """Rows without a valid page are left out and noted."""
    f = Filled(2, 64, 16, [70, 40], seed=11)
    f.cache.table[0, 2] = -1
    f.cache.table[1, 0] = 1 << 20
    q = torch.randn(2, 4, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).to(io)
    out = f.cache.attention(f.layer, q)
    with pytest.raises(dec.DecError, match="index"):
        f.cache.sync_status()
    for s, gone in ((0, slice(32, 48)), (1, slice(0, 16))):
        f.k[s], f.v[s] = (np.delete(x, np.arange(*gone.indices(100)), 1) for x in (f.k[s], f.v[s]))
    f.check(q, out, [0, 1])


def test_attention_over_a_nan_block_is_nan():
    """A block with a NaN scale gives NaN to the queries that see it, and to no other."""
    for half in (0, 1):                                   # of K, of V
        f = Filled(1, 64, 16, [40, 40], seed=12, spare=0)
        page = int(f.cache.table[0, 1])
        _, scales = f.pages.parts(f.pool[1, page])
        scales[half][0, 0] = np.nan
        f.cache.pool.copy_(torch.from_numpy(f.pool))
        q = torch.randn(2, 1, 64, device="cuda")
        for io in (torch.float32, torch.bfloat16):
            out = f.cache.attention(1, q.to(io))
            assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())
            out = f.cache.attention(1, q.to(io), window=8)    # the rows behind it alone
            assert bool(out.isfinite().all())


def test_offsets_past_32_bits():
    """A page whose bytes lie past 4 GiB: written, read and attended."""
    nkv, hd, R = 32, 128, 1024                             # 8.4 MB a page
    n_pages = 530
    c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt="q8", n_pages=n_pages, n_seqs=1, max_pages=2)
    assert n_pages * c.page_bytes > 1 << 32
    c.table[0] = ints([n_pages - 1, 515])
    c.lens.fill_(1030)
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(6, nkv, hd, device="cuda", generator=g) for _ in range(2))
    at = [1024, 1025, 1026, 1027, 1028, 1029]
    c.append(0, k, v, seqs=ints([0] * 6), positions=ints(at))
    kk, vv = c.read(0, ints([0] * 6), ints(at))
    assert (kk - k).abs().max() <= k.abs().max() / 127 and (vv - v).abs().max() <= v.abs().max() / 127
    q = torch.randn(1, nkv, hd, device="cuda", generator=g)
    out = c.attention(0, q, window=6)
    f = Filled.__new__(Filled)
    f.pages, f.k, f.v = ref.Pages8(nkv, hd, R), [f64(kk).transpose(1, 0, 2)], [f64(vv).transpose(1, 0, 2)]
    f.check(q, out, [0])


# ---- pages ---------------------------------------------------------------------


def test_fork_release_and_compact_keep_blocks():
    """Forked sequences grow apart, pages move: the rows stay what they were."""
    c = kv.KVCache(n_layers=2, n_kv_heads=2, head_dim=64, page_rows=32, fmt="q8", n_pages=24, n_seqs=6, max_pages=5)
    g = torch.Generator(device="cuda").manual_seed(9)
    c.extend(ints([0, 1]), ints([70, 20]))
    k, v = (torch.randn(90, 2, 64, device="cuda", generator=g) for _ in range(2))
    seqs, pos = ints([0] * 70 + [1] * 20), ints(list(range(70)) + list(range(20)))
    for layer in range(2):
        c.append(layer, k, v, seqs=seqs, positions=pos)
    had = [c.read(layer, seqs, pos) for layer in range(2)]
    c.fork(ints([0, 0, 1]), ints([2, 3, 4]))
    for s in (0, 2, 3):                                   # each its own next row, larger than all before
        c.extend(ints([s]))
        x = torch.full((1, 2, 64), 100.0 * (s + 1), device="cuda")
        c.append(1, x, x, seqs=ints([s]))
    c.sync_status()
    for s in (0, 2, 3):
        kk, _ = c.read(1, ints([s] * 71), ints(range(71)))
        step = 2.0 ** ref.scale_exponent(100.0 * (s + 1))
        assert bool((kk[70] - 100.0 * (s + 1)).abs().max() <= step / 2)
        assert torch.equal(kk[:64], had[1][0][:64])       # shared blocks are untouched
        assert bool((kk[64:70] - k[64:70]).abs().max() <= step)
    c.release(ints([1, 3]))
    c.compact()
    c.sync_status()
    for layer in range(2):
        kk, vv = c.read(layer, ints([2] * 64 + [4] * 20), ints(list(range(64)) + list(range(20))))
        for i, got in enumerate((kk, vv)):
            assert torch.equal(got[:64], had[layer][i][:64]) and torch.equal(got[64:], had[layer][i][70:])
