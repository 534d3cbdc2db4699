"""Long lists of rows written to 8-bit pages, byte for byte: those whose rows are looked through by every CTA, those
that are noted first, CTAs that take all the entries they can, heads that take several turns of a CTA's warps."""
import numpy as np
import pytest

from test_gpu_kv8 import Walk, ints
from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv, rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def begun(w, plan):
    """Blocks that hold nothing yet get some scale, as if they had been begun before."""
    for s, b in {(s, p // 16) for s, p in plan if s >= 0} - set(w.live):
        for part in w.p.parts(w.pool[w.layer, w.table[s, b * 16 // w.R]])[1]:
            part[:, b * 16 % w.R // 16] = 2.0 ** -6
    w.cache.pool.copy_(torch.from_numpy(w.pool))


def plan_of(rng, n, n_seqs, order, padding=True):
    starts = rng.integers(0, 60, n_seqs)
    plan = [(s, int(starts[s]) + i) for s in range(n_seqs) for i in range(-(-n // n_seqs))][:n]
    if order == "across":
        plan.sort(key=lambda x: (x[1], x[0]))
    if order == "shuffled":
        plan = [plan[i] for i in rng.permutation(n)]
    if padding:
        plan[n // 3], plan[n - 1] = (-1, 7), (-5, 0)
    return plan


@pytest.mark.parametrize("nkv,hd,R,io", [(9, 64, 64, torch.float32), (1, 128, 48, torch.bfloat16)])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 4096, 4111, 6001])
@pytest.mark.parametrize("order", ["runs", "across", "shuffled"])
def test_long_lists_in_any_order(n, order, nkv, hd, R, io):
    w = Walk(nkv, hd, R, 8, -(-(-(-n // 8) + 60) // R), seed=n + nkv)
    for turn in range(2):
        plan = plan_of(w.rng, n, 8, order)
        begun(w, plan)
        w.append(plan, io, 2.0 ** (turn - 1))
        w.check()
        w.pool[:] = w.cache.pool.cpu().numpy()


def test_one_head_s_blocks_on_every_turn():
    """An odd number of heads above a CTA's warps, which share them with other CTAs."""
    w = Walk(21, 64, 16, 40, 4, seed=3)
    plan = plan_of(w.rng, 40 * 4, 40, "runs")
    begun(w, plan)
    w.append(plan, torch.bfloat16, 1.0)
    w.check()


def test_bad_rows_of_a_long_list_are_skipped():
    w = Walk(2, 64, 16, 4, 2, seed=1)
    before = w.cache.pool.clone()
    w.cache.table[2, 1] = -1
    w.cache.table[3, 0] = 99
    many = torch.ones(1800, 2, 64, device="cuda")
    for seqs, positions in (([4, -1, 70000], [0, 0, 0]), ([2, 3, -7], [17, 4, 3]), ([0, 1, 2], [32, -1, 1 << 30])):
        w.cache.append(1, many, many, seqs=ints(seqs * 600), positions=ints(positions * 600))
        with pytest.raises(dec.DecError, match="index"):
            w.cache.sync_status()
        assert torch.equal(w.cache.pool, before)


def test_long_appends_of_two_streams_share_nothing():
    """Calls on other layers, and on other blocks of a layer, may overlap."""
    each = 160
    w = Walk(2, 64, 64, 16, 4, layers=2, layer=1, seed=5)
    mine, other = ([(s, i) for s in r for i in range(each)] for r in (range(8), range(8, 16)))
    (t, x), (u, y) = w.rows(8 * each, torch.float32, 1.0), w.rows(8 * each, torch.float32, 1.0)
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
    live, w.live, w.layer = w.live, {}, 0
    w.note(mine, y)
    got = w.cache.pool.cpu().numpy()
    for layer, blocks in ((1, live), (0, w.live)):
        for (s, b), rows in blocks.items():
            page, block = w.table[s, b * 16 // 64], b * 16 % 64 // 16
            for want, have in zip(zip(*w.p.parts(w.pool[layer, page])), zip(*w.p.parts(got[layer, page]))):
                assert np.array_equal(want[1][:, block], have[1][:, block])
                at = 16 * block + np.array(sorted(rows))
                assert np.array_equal(want[0][:, at], have[0][:, at])


@pytest.mark.parametrize("rotated", [False, True])
def test_long_lists_in_the_debug_build(rotated):
    """The index checks of the debug build find nothing, and its bytes are the release build's."""
    rng, pools = np.random.default_rng(8), []
    plan = plan_of(rng, 1500, 6, "shuffled")
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(1500, 3, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1500, 6, 128, device="cuda", generator=g).bfloat16()
    for lib in (dec.LIB_PATH, tld_build.build(debug=True)):
        c = kv.KVCache(n_layers=1, n_kv_heads=3, head_dim=128, page_rows=16, fmt="q8", n_pages=140, n_seqs=6, max_pages=23,
                       lib_path=lib)
        c.pool.zero_()
        c.extend(n_new=ints([311] * 6))
        seqs, pos = ints([s for s, _ in plan]), ints([p for _, p in plan])
        out = torch.zeros_like(q)
        if rotated:
            c.append_rotated(0, rope.Rotary(128, lib_path=lib), q, k, v, seqs=seqs, positions=pos, q_out=out)
        else:
            c.append(0, k, v, seqs=seqs, positions=pos)
        c.sync_status()
        pools.append((c.pool, out))
    assert all(torch.equal(a, b) for a, b in zip(*pools))
