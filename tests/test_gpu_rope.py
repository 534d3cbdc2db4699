"""Rotary positions on the GPU against their 64-bit statement, alone and on the way into a cache.

Tolerances.  The angle is off by 2^-25 of half a turn (its rounding to fp32) and by
2^-32 turns for what is cut off before, pi * 2^-25 + 2 pi * 2^-32 < 2^-23.2; cos and
sin are good to 2 ulp (2^-23 at most), the magnitude's product and the pair's
products and sum take 2^-24 of the pair's size each: in all below 2^-21 of
magnitude * (|a| + |b|), plus half a step of the result's type (bf16 2^-8, fp32 2^-24).
The frequencies of both sides are doubles, good to 2^-50 with their powers: at position p
an angle may differ by p * 2^-50, and by p * 2^-52 for the statement's own product.
"""
import numpy as np
import pytest

import kv8_reference as ref
import kv_reference as ref4
from test_gpu_kv8 import Filled, f64, ints
from test_gpu_kv_cache import Filled as OtherFilled
from transformer_layer_decode_gb300 import dec, kv, rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def limit(x, y, positions, freq, magnitude, layout, io):
    rot, size = 2 * len(freq), np.zeros(x.shape)
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    size[..., a] = size[..., b] = abs(magnitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    far = np.abs(np.asarray(positions, np.float64))[:, None, None] * 1.25 * 2.0 ** -50
    tol = size * (2.0 ** -21 + far)
    return tol + (np.abs(y) + tol) * (2.0 ** -8 if io == torch.bfloat16 else 2.0 ** -24) + 1e-38


def rows(shape, io, seed=0):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(io)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (128, 64), (128, 32), (80, 80), (80, 20), (96, 24), (128, 2),
                                    (8, 8), (8, 6), (256, 250), (1024, 1024), (72, 64)])
@pytest.mark.parametrize("n,heads", [(1, 1), (7, 3), (65, 8)])
def test_rotate(io, layout, hd, rot, n, heads):
    r = rope.Rotary(hd, rot_dim=rot, layout=layout, theta=5e5)
    x = rows((n, heads, hd), io, seed=hd + rot)
    rng = np.random.default_rng(n)
    positions = rng.integers(0, 10000, n)
    freq, m = ref.frequencies(rot, theta=5e5)
    for backward in (False, True):
        y = r.rotate(x, ints(positions), backward=backward)
        want = ref.rotate(f64(x), positions, freq, m, layout, backward)
        assert (np.abs(f64(y) - want) <= limit(f64(x), want, positions, freq, m, layout, io)).all()
        assert torch.equal(y[..., rot:], x[..., rot:])
        z = x.clone()                                     # in place: the same bits
        assert r.rotate(z, ints(positions), out=z, backward=backward) is z and torch.equal(z, y)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=8.0, context=2048))])
def test_scalings(scaling, kw):
    r = rope.Rotary(128, rot_dim=96, scaling=scaling, **kw)
    x, positions = rows((50, 4, 128), torch.float32), np.arange(50) * 327
    freq, m = ref.frequencies(96, scaling=scaling, **kw)
    want = ref.rotate(f64(x), positions, freq, np.float64(np.float32(m)), "half")
    assert (np.abs(f64(r.rotate(x, ints(positions))) - want) <= limit(f64(x), want, positions, freq, m, "half", torch.float32)).all()
    assert abs(r.magnitude - m) < 1e-6


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout):
    """Positions up to 2^31 - 1: as exact as near ones."""
    freq = np.array([1.0, 0.5, 3.0e-3, 2.0 ** -20, 6.0, 0.0, -1.0, 1e-9])
    r = rope.Rotary(16, layout=layout, frequencies=freq, magnitude=1.25)
    positions = np.array([0, 1, 2, 1000, 99999, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, 1234567890])
    x = rows((len(positions), 2, 16), torch.float32, 3)
    want = ref.rotate(f64(x), positions, freq, 1.25, layout)
    got = f64(r.rotate(x, ints(positions)))
    # (the statement's own product position * frequency rounds to 2^-53 of itself)
    assert (np.abs(got - want) <= limit(f64(x), want, positions * 6, freq, 1.25, layout, torch.float32)).all()


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hd,rot", [(128, 64), (64, 20)])
def test_rows_that_are_skipped_and_strides(io, hd, rot):
    r = rope.Rotary(hd, rot_dim=rot)
    wide = rows((9, 7, hd), io)
    x, out = wide[:, 1:5], torch.full((9, 6, hd), 2.0, device="cuda", dtype=io)
    positions = np.array([3, -1, 0, 5, 1 << 20, -9, 7, 8, -1])
    r.rotate(x, ints(positions), out=out[:, 2:])
    live = positions >= 0
    freq, m = ref.frequencies(rot)
    want = ref.rotate(f64(x), positions, freq, m, "half")
    tol = limit(f64(x), want, positions, freq, m, "half", io)
    assert (np.abs(f64(out[:, 2:]) - want) <= tol)[live].all()
    assert bool((out[:, :2] == 2).all()) and bool((out[~torch.from_numpy(live)] == 2).all())
    made = r.rotate(x, ints(positions))
    assert torch.equal(made[live], out[:, 2:][live]) and not made[~torch.from_numpy(live)].any()
    assert torch.equal(r.rotate(x), r.rotate(x, ints(range(9))))   # without positions: 0, 1, ...
    inside = wide.clone()                                          # in place among other heads
    r.rotate(inside[:, 1:5], ints(positions), out=inside[:, 1:5])
    assert torch.equal(inside[live][:, 1:5], made[live]) and torch.equal(inside[:, 5:], wide[:, 5:])
    assert torch.equal(inside[~torch.from_numpy(live)], wide[~torch.from_numpy(live)])
    assert r.rotate(x[:0]).shape == (0, 4, hd)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,heads,hd,rot", [(8000, 5, 64, 64), (3, 700, 64, 64), (1, 4000, 64, 64), (310, 1300, 64, 64),
                                            (320, 70, 1024, 512), (20011, 1, 8, 8), (1300, 3, 96, 42)])
def test_many_rows_and_heads(io, n, heads, hd, rot):
    """Every way of cutting the rows between CTAs: rows together, heads apart, both."""
    r = rope.Rotary(hd, rot_dim=rot, layout="half")
    x = rows((n, heads, hd), io)
    positions = (np.arange(n) * 13) % 5000
    got = r.rotate(x, ints(positions))
    freq, m = ref.frequencies(rot)
    want = ref.rotate(f64(x), positions, freq, m, "half")
    assert (np.abs(f64(got) - want) <= limit(f64(x), want, positions, freq, m, "half", io)).all()


def test_on_another_stream_and_in_a_graph():
    r = rope.Rotary(128)
    x, positions = rows((600, 4, 128), torch.bfloat16), ints(range(600))
    want = r.rotate(x, positions)
    side, out = torch.cuda.Stream(), torch.zeros_like(x)
    side.wait_stream(torch.cuda.current_stream())
    r.rotate(x, positions, out=out, stream=side)
    made = r.rotate(x, positions, stream=side)
    by_handle = r.rotate(x, positions, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(made, want) and torch.equal(by_handle, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = r.rotate(x, positions)
    x.copy_(rows(x.shape, torch.bfloat16, 9))
    positions.add_(7)
    graph.replay()
    assert torch.equal(kept, r.rotate(x, positions))


@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 64), ("half", 20)])
def test_gradient(layout, rot):
    """backward is the transposed rotation: the formula's, and what differences give (the rotation is linear,
    so a difference over any step is the derivative, up to the two results' roundings)."""
    r = rope.Rotary(64, rot_dim=rot, layout=layout, scaling="yarn", factor=4.0, context=2048)
    x, dy, e = (rows((40, 2, 64), torch.float32, s) for s in (1, 2, 3))
    positions = ints(np.arange(40) * 51)
    dx = f64(r.rotate(dy, positions, backward=True))
    along = (f64(r.rotate(x + e, positions)) - f64(r.rotate(x, positions)))
    step = f64(x + e) - f64(x)
    size = 2 * r.magnitude * (np.abs(f64(dy)).sum() * (np.abs(f64(x)).max() + np.abs(f64(e)).max()))
    assert abs((dx * step).sum() - (f64(dy) * along).sum()) <= 4 * 2.0 ** -21 * size
    freq, m = ref.frequencies(rot, scaling="yarn", factor=4.0, context=2048)
    want = ref.rotate(f64(dy), np.arange(40) * 51, freq, m, layout, True)
    assert (np.abs(dx - want) <= limit(f64(dy), want, np.arange(40) * 51, freq, m, layout, torch.float32)).all()


def test_refusals():
    r = rope.Rotary(64)
    x = rows((4, 2, 64), torch.float32)
    for bad in (x.half(), x.cpu(), x[..., :32], x.transpose(0, 1).contiguous().transpose(0, 1), x[:, :, None], x.double(),
                x[:, :0]):
        with pytest.raises(ValueError, match="x:"):
            r.rotate(bad)
    for bad in (ints([0, 1, 2]), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int32),
                ints(range(8))[::2]):
        with pytest.raises(ValueError, match="positions"):
            r.rotate(x, bad)
    with pytest.raises(ValueError, match="out"):
        r.rotate(x, out=x.bfloat16())
    with pytest.raises(ValueError, match="out"):
        r.rotate(x, out=torch.empty(4, 3, 64, device="cuda"))
    buf = torch.zeros(9, 2, 64, device="cuda")
    with pytest.raises(dec.DecError, match="overlap"):
        r.rotate(buf[:4], out=buf[3:7])
    odd = torch.zeros(1 + 4 * 128, device="cuda")[1:].view(4, 2, 64)
    with pytest.raises(dec.DecError, match="aligned"):
        r.rotate(odd)
    c = kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=128, fmt="q8", n_pages=2, n_seqs=4, max_pages=1)
    k = torch.zeros(4, 2, 128, device="cuda")
    with pytest.raises(dec.DecError, match="head_dim"):
        c.append_rotated(0, r, None, k, k)
    r = rope.Rotary(128)
    with pytest.raises(ValueError, match="q"):
        c.append_rotated(0, r, k[:3], k, k)
    with pytest.raises(ValueError, match="q"):
        c.append_rotated(0, r, k.bfloat16(), k, k)
    with pytest.raises(ValueError, match="q_out"):
        c.append_rotated(0, r, None, k, k, q_out=k)
    with pytest.raises(dec.DecError, match="overlap"):
        c.append_rotated(0, r, torch.ones_like(k), k, k.clone(), q_out=k)
    with pytest.raises(ValueError, match="layer"):
        c.append_rotated(1 << 32, r, None, k, k)


# ---- on the way into a cache -----------------------------------------------------


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("layout,rot,hd,nkv,heads,R", [("half", 128, 128, 2, 6, 32), ("interleaved", 64, 64, 3, 3, 16),
                                                        ("half", 32, 64, 1, 4, 64), ("half", 20, 128, 4, 4, 16),
                                                        ("interleaved", 50, 128, 2, 10, 48)])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_append_rotated(io, fmt, layout, rot, hd, nkv, heads, R, n):
    """The bytes of a rotation in fp32 and then an append, and the queries of a rotation alone."""
    width = -(-(n + 30) // R)
    r = rope.Rotary(hd, rot_dim=rot, layout=layout, scaling="linear", factor=2.0)

    def make():
        c = kv.KVCache(n_layers=2, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=3 * width + 1, n_seqs=3,
                       max_pages=width)
        c.pool.zero_()
        c.table.copy_(ints(np.arange(3 * width).reshape(3, width)))
        c.lens.fill_(width * R)
        return c

    a, b = make(), make()
    k, v, q = rows((n, nkv, hd), io, 1), rows((n, nkv, hd), io, 2), rows((n, heads, hd), io, 3)
    plan = [(t % 3, 17 + t // 3) for t in range(n)]
    if n > 30:
        plan[5], plan[n - 1] = (-1, 0), (-2, 4)
    seqs, positions = ints([s for s, _ in plan]), ints([p for _, p in plan])
    live = seqs >= 0
    out = torch.full_like(q, 4.0)
    assert a.append_rotated(1, r, q, k, v, seqs=seqs, positions=positions, q_out=out) is out
    turned = r.rotate(k.float(), positions)
    b.append(1, turned, v.float(), seqs=seqs, positions=positions)
    a.sync_status()
    b.sync_status()
    assert torch.equal(a.pool, b.pool)
    want = r.rotate(q, positions)
    assert torch.equal(out[live], want[live]) and bool((out[~live] == 4).all())
    assert torch.equal(a.append_rotated(1, r, q, k, v, seqs=seqs, positions=positions)[live], want[live])


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("layout,rot,hd,nkv,heads,R,n", [
    ("half", 128, 128, 8, 32, 64, 2100), ("interleaved", 64, 64, 5, 40, 16, 3301), ("half", 20, 128, 3, 1, 48, 2750),
    ("half", 32, 64, 17, 2, 32, 1201), ("interleaved", 128, 128, 8, 2, 16, 4111)])
def test_append_many_rotated(io, fmt, layout, rot, hd, nkv, heads, R, n):
    """Rows enough for several turns of a CTA, and queries enough for a launch of their own or not."""
    test_append_rotated(io, fmt, layout, rot, hd, nkv, heads, R, n)


@pytest.mark.parametrize("fmt", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("listed", [False, True])
def test_steps_of_many_sequences_in_a_graph(fmt, listed):
    """Many queries, of one row each and of a list, whose lists, rows and pages the kernels just before change."""
    n, heads, nkv, hd, R, steps = 2100, 32, 2, 128, 16, 3
    r = rope.Rotary(hd)

    def make():
        c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=2 * n, n_seqs=n, max_pages=2)
        c.pool.zero_()
        c.extend(n_new=ints([14 + i % 3 for i in range(n)]))
        return c

    a, b = make(), make()
    seqs, pos = ints(range(n)), ints([0] * n)
    q, k, v = (rows((n, h, hd), torch.bfloat16, h) for h in (heads, nkv, nkv + 1))
    v = v[:, :nkv].contiguous()
    out = torch.empty_like(q)

    def step():
        q.add_(0.25), k.mul_(1.5), v.mul_(-1.25)
        a.extend()
        torch.sub(a.lens, 1, out=pos)
        if listed:
            seqs.copy_(seqs.flip(0))
            pos.copy_(pos[seqs])
            a.append_rotated(0, r, q, k, v, seqs=seqs, positions=pos, q_out=out)
        else:
            a.append_rotated(0, r, q, k, v, q_out=out)

    def same():
        b.extend()
        torch.cuda.synchronize()
        b.append_rotated(0, r, None, k, v, seqs=seqs, positions=pos if listed else b.lens - 1)
        torch.cuda.synchronize()
        assert torch.equal(a.pool, b.pool)
        assert torch.equal(out, r.rotate(q, pos))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
        same()
    a.sync_status()
    b.sync_status()


def test_one_projection_s_rows_in_place():
    """q, k and v as slices of one tensor, q rotated where it lies; and keys alone."""
    r = rope.Rotary(64)
    for fmt in ("q8", "q4", "bf16"):
        c, d = (kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, page_rows=16, fmt=fmt, n_pages=8, n_seqs=5, max_pages=1)
                for _ in range(2))
        for x in (c, d):
            x.pool.zero_()
            x.extend(n_new=ints([1, 2, 3, 4, 5]))
        qkv = rows((5, 12, 64), torch.bfloat16, 5)
        was = qkv.clone()
        c.append_rotated(0, r, qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], q_out=qkv[:, :8])
        assert torch.equal(qkv[:, 8:], was[:, 8:])
        assert torch.equal(qkv[:, :8], r.rotate(was[:, :8], ints(range(5))))
        assert d.append_rotated(0, r, None, was[:, 8:10], was[:, 10:]) is None
        c.sync_status()
        assert torch.equal(c.pool, d.pool)


def test_rotated_append_skips_what_is_bad():
    r = rope.Rotary(64)
    for fmt in ("q8", "q4", "bf16"):
        c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, fmt=fmt, n_pages=4, n_seqs=3, max_pages=1)
        c.pool.fill_(7)
        k, q = rows((4, 1, 64), torch.float32), rows((4, 2, 64), torch.float32)
        out = torch.full_like(q, 9.0)
        c.append_rotated(0, r, q, k, k, seqs=ints([0, 5, -1, 1]), positions=ints([16, 0, 0, 3]), q_out=out)
        with pytest.raises(dec.DecError, match="index"):
            c.sync_status()
        assert bool((out == 9).all()) and bool((c.pool == 7).all())   # (no sequence has a page)


# ---- together ---------------------------------------------------------------------


@pytest.mark.parametrize("fmt", ["q8", "q4", "bf16"])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_a_decode_loop_in_a_graph(fmt, io):
    """A prompt, then steps of extend, append_rotated and attention, captured once and replayed: what each step
    gives is attention over the rows as they can be read back, keys rotated by their positions."""
    n, heads, nkv, hd, R, steps = 5, 8, 2, 64, 16, 40
    r = rope.Rotary(hd, layout="interleaved", scaling="yarn", factor=4.0, context=64)
    c = kv.KVCache(n_layers=1, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_pages=40, n_seqs=n, max_pages=6)
    prompt = [3, 0, 17, 32, 9]
    c.extend(n_new=ints(prompt))
    total = sum(prompt)
    k, v = rows((total, nkv, hd), io, 1), rows((total, nkv, hd), io, 2)
    seqs = ints([s for s, m in enumerate(prompt) for _ in range(m)])
    pos = ints([i for m in prompt for i in range(m)])
    c.append_rotated(0, r, None, k, v, seqs=seqs, positions=pos)
    q, k1, v1 = rows((n, heads, hd), io), rows((n, nkv, hd), io), rows((n, nkv, hd), io)
    turned, out = torch.empty_like(q), torch.empty_like(q)
    lens0, table0, refs0, pool0 = (t.clone() for t in (c.lens, c.table, c.refs, c.pool))

    def step():
        c.extend()
        c.append_rotated(0, r, q, k1, v1, q_out=turned)
        c.attention(0, turned, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                            # (workspaces and the kernels' first use)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, was in ((c.lens, lens0), (c.table, table0), (c.refs, refs0), (c.pool, pool0)):
        t.copy_(was)
    for i in range(steps):
        for t, seed in ((q, 10), (k1, 11), (v1, 12)):
            t.copy_(rows(t.shape, io, seed + 7 * i) * (1 + i % 5))
        graph.replay()
        if i % 13 and i != steps - 1:
            continue
        c.sync_status()
        lens = c.lens.cpu().numpy()
        assert (lens == np.array(prompt) + i + 1).all()
        turned_want = r.rotate(q, c.lens - 1)
        assert torch.equal(turned, turned_want)
        # (each format's tolerances are those of its own tests, which state them)
        kind, pages = (Filled, ref.Pages8(nkv, hd, R)) if fmt == "q8" else (OtherFilled, ref4.Pages(fmt, nkv, hd, R))
        f = kind.__new__(kind)
        f.pages, f.k, f.v = pages, [], []
        for s in range(n):
            m = int(lens[s])
            kk, vv = c.read(0, ints([s] * m), ints(range(m)))
            f.k.append(f64(kk).transpose(1, 0, 2))
            f.v.append(f64(vv).transpose(1, 0, 2))
        f.check(turned, out, range(n), what=(fmt, i))
