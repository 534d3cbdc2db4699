"""8-bit blocks that are not begun at their first row, on pages that held something else: their scale is their own."""
import numpy as np
import pytest

import kv8_reference as ref
from transformer_layer_decode_gb300 import dec, kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


def append_and_compare(c, p, plan, *, layer, positions=True, seed=0):
    """Rows of `plan` [(sequence, position)] of one layer, whose pages have never held any: bytes and values."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (2, len(plan), p.h, p.d)).astype(np.float32)
    table = c.table.cpu().numpy()
    t = torch.from_numpy(x).cuda()
    c.append(layer, t[0], t[1], seqs=ints([s for s, _ in plan]), positions=ints([r for _, r in plan]) if positions else None)
    c.sync_status()
    pool, by_block = c.pool.cpu().numpy()[layer], {}
    for i, (s, r) in enumerate(plan):
        by_block.setdefault((s, r // 16), {})[r % 16] = x[:, i]
    for (s, b), rows in by_block.items():
        page, block = np.zeros(p.page_bytes, np.uint8), b * 16 % p.R // 16
        p.write(page, block, rows)
        got, want = p.parts(pool[table[s, b * 16 // p.R]]), p.parts(page)
        for half in range(2):
            assert np.array_equal(got[1][half][:, block], want[1][half][:, block]), (s, b, half)
            at = [16 * block + r for r in rows]
            assert np.array_equal(got[0][half][:, at], want[0][half][:, at]), (s, b, half)
            before = got[0][half][:, 16 * block:16 * block + min(rows)]  # what no one wrote reads as 0
            assert (before == 128).all(), (s, b, half)


@pytest.mark.parametrize("junk", [0xFF, 0x7E, 0x46])   # scales of NaN, 2^125 and 12688 where no one wrote
@pytest.mark.parametrize("hd,nkv,R", [(64, 1, 16), (128, 3, 48), (64, 8, 128)])
@pytest.mark.parametrize("n", [1, 30, 700])
def test_rows_of_a_window_alone(junk, hd, nkv, R, n):
    """The last n rows of prompts, written at once (short lists and long ones), and then a decode step's."""
    p, n_seqs, lens = ref.Pages8(nkv, hd, R), 4, [n + 5, n + 16, n, n + 27]
    width = -(-(n + 30) // R)
    c = kv.KVCache(n_layers=3, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt="q8", n_pages=4 * width + 1, n_seqs=n_seqs,
                   max_pages=width)
    c.pool.fill_(junk)
    c.extend(n_new=ints(lens))
    free = sorted(set(range(4 * width + 1)) - set(c.table.cpu().numpy().ravel().tolist()))
    assert bool((c.pool[:, free] == junk).all())       # (pages that no one was given stay as they are)
    for layer in (2, 0):
        append_and_compare(c, p, [(s, m - n + i) for s, m in enumerate(lens) for i in range(n)], layer=layer, seed=layer)
    c.release()
    c.pool.fill_(junk)
    c.extend(n_new=ints([m - n for m in lens]))          # a block's beginning is skipped, its next row written
    c.extend()
    append_and_compare(c, p, [(s, m - n) for s, m in enumerate(lens)], layer=1, positions=False)


def test_a_page_s_next_owner():
    """Rows of another sequence, much larger, before; the pages go round by release and extend, in a graph too."""
    p = ref.Pages8(2, 64, 32)
    c = kv.KVCache(n_layers=1, n_kv_heads=2, head_dim=64, page_rows=32, fmt="q8", n_pages=6, n_seqs=2, max_pages=3)
    n_new, seqs, pos = ints([70, 0]), ints([0] * 70), ints(range(70))
    large = torch.full((70, 2, 64), 1e20, device="cuda")
    swap = ints([0, 70])

    def turn():
        c.extend(n_new=n_new)
        c.append(0, large, large, seqs=seqs, positions=pos)
        c.release(seqs[:1])
        c.extend(n_new=swap)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn()
    torch.cuda.current_stream().wait_stream(side)
    append_and_compare(c, p, [(1, i) for i in range(5, 70)], layer=0)
    c.release()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for seed in range(3):
        graph.replay()
        append_and_compare(c, p, [(1, i) for i in range(21, 70)], layer=0, seed=seed)
        c.release()
    c.sync_status()


def test_a_new_cache_without_extend():
    """Pages that the caller puts into the table of a cache made here, on memory that held something."""
    p = ref.Pages8(2, 64, 32)
    junk = torch.full((2, 64, p.page_bytes), 0x7E, dtype=torch.uint8, device="cuda")
    del junk  # (the allocator hands it out again)
    c = kv.KVCache(n_layers=2, n_kv_heads=2, head_dim=64, page_rows=32, fmt="q8", n_pages=64, n_seqs=2, max_pages=3)
    c.table.copy_(ints([[5, 0, 63], [7, 8, 9]]))
    c.lens.fill_(80)
    code_bytes = p.code_bytes
    halves = c.pool.view(2, 64, 2, p.half_bytes)
    halves[..., :code_bytes].fill_(128)                # (rows that no one wrote hold anything; the comparison wants 0)
    append_and_compare(c, p, [(s, i) for s in range(2) for i in range(9, 80)], layer=1)


def test_an_extend_that_is_refused_changes_nothing():
    c = kv.KVCache(n_layers=2, n_kv_heads=2, head_dim=64, page_rows=16, fmt="q8", n_pages=4, n_seqs=3, max_pages=4)
    c.extend(ints([0]), ints([20]))
    c.pool.random_(0, 256)
    was = [t.clone() for t in (c.pool, c.table, c.lens, c.refs)]
    for n_new in ([40, 30], [30, -1]):
        c.extend(ints([1, 2]), ints(n_new))
        with pytest.raises(dec.DecError):
            c.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(was, (c.pool, c.table, c.lens, c.refs)))
    c.extend(ints([0]), ints([12]))                     # no page more: nothing to clear
    c.sync_status()
    assert torch.equal(c.pool, was[0])
