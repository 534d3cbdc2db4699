"""Calls of the paged cache in the circumstances that its documentation allows: host threads, streams, captures
that others begin, the largest sizes, pages and lengths out of range."""
import ctypes
import threading

import numpy as np
import pytest

from transformer_layer_decode_gb300 import dec, kv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


def filled(fmt, nkv, hd, R, lens, *, spare=3, seed=0, layers=1, room=0):
    """A cache with sequences of these lengths, all rows written."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    width = max(1, -(-room // R), max(-(-n // R) for n in lens))
    c = kv.KVCache(n_layers=layers, n_kv_heads=nkv, head_dim=hd, page_rows=R, fmt=fmt, n_seqs=len(lens),
                   n_pages=sum(-(-n // R) for n in lens) + spare, max_pages=width)
    c.extend(None, ints(lens))
    seqs = ints([s for s, n in enumerate(lens) for _ in range(n)])
    pos = ints([j for n in lens for j in range(n)])
    for layer in range(layers):
        k, v = (torch.randn(len(seqs), nkv, hd, device="cuda", generator=gen) for _ in range(2))
        c.append(layer, k, v, seqs=seqs, positions=pos)
    c.sync_status()
    return c


def in_threads(*works):
    errors = []

    def run(work):
        try:
            work()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attention_of_threads_on_one_stream(fmt):
    """Units cut into parts, which the second launch of a call joins: with another call's first launch between
    the two it would join that one's."""
    c = filled(fmt, 2, 64, 16, [3000, 2500])
    n = 6
    qs = [torch.randn(2, 4, 64, device="cuda") for _ in range(n)]
    want = [c.attention(0, q).clone() for q in qs]
    outs = [[] for _ in qs]

    def work(i):
        for _ in range(300):
            outs[i].append(c.attention(0, qs[i]))

    torch.cuda.synchronize()
    in_threads(*(lambda i=i: work(i) for i in range(n)))
    torch.cuda.synchronize()
    for i in range(n):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    c.sync_status()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_pages_of_threads_on_one_stream(fmt):
    """Threads that fork, extend, release and compact one cache over and over: every plan is carried out by its
    own call, so at the end the tables name each page as often as it is counted, and the forks hold their
    parents' rows."""
    lens = [40, 0, 0, 100, 0, 0, 7, 0, 0]
    c = filled(fmt, 1, 64, 16, lens, spare=60, room=160, layers=2)
    torch.cuda.synchronize()

    def work(parent):
        parents, children = ints([parent, parent]), ints([parent + 1, parent + 2])
        for i in range(60):
            c.fork(parents, children)
            c.extend(children)
            if i < 59:
                c.release(children)
            if i % 7 == parent:
                c.compact()

    in_threads(*(lambda p=p: work(p) for p in (0, 3, 6)))
    c.sync_status()
    assert c.lens.tolist() == [lens[p] + more for p in (0, 3, 6) for more in (0, 1, 1)]
    table = c.table.cpu().numpy()
    assert np.array_equal(np.bincount(table[table >= 0], minlength=c.refs.numel()), c.refs.cpu().numpy())
    for parent in (0, 3, 6):
        pos = ints(range(lens[parent]))
        for layer in range(2):
            rows = [c.read(layer, torch.full_like(pos, s), pos) for s in (parent, parent + 1, parent + 2)]
            for k, v in rows[1:]:
                assert torch.equal(k, rows[0][0]) and torch.equal(v, rows[0][1])
    c.sync_status()


@pytest.mark.parametrize("fmt,room", [("bf16", 64), ("q4", 64), ("bf16", 4096), ("q4", 4096)])
def test_skipped_rows_of_a_result_made_here_are_zero(fmt, room):
    """A length out of range skips its sequence, in a list or not: zeros, whatever the memory held before."""
    c = filled(fmt, 2, 64, 16, [30, 40, 50], room=room)
    q = torch.randn(3, 4, 64, device="cuda")
    want = c.attention(0, q)
    c.lens[1] = room + 1
    c.lens[2] = -1
    want[1:] = 0
    for seqs in (None, ints([0, 1, 2])):
        torch.cuda.synchronize()
        junk = [torch.full_like(q, float("nan")) for _ in range(64)]   # what the allocator hands out next
        del junk
        got = c.attention(0, q, seqs=seqs)
        with pytest.raises(dec.DecError, match="index"):
            c.sync_status()
        assert torch.equal(got, want)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("fmt,room", [("bf16", 16), ("q4", 16), ("bf16", 4096), ("q4", 4096)])
def test_the_most_queries(fmt, room, listed):
    """65536 sequences at once, short of rows or not (kernels that count, and that do not): the rows are pages
    that all share, so the results come in kinds."""
    n, hd, R = 65536, 64, 16
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=hd, page_rows=R, fmt=fmt, n_pages=3, n_seqs=n, max_pages=room // R)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(3 * R, 1, hd, device="cuda", generator=gen) for _ in range(2))
    c.lens[:3] = R
    c.table[:3, 0] = ints([0, 1, 2])
    c.append(0, k, v, seqs=ints(np.repeat(range(3), R)), positions=ints(np.tile(range(R), 3)))
    kind = torch.arange(n, device="cuda") % 48
    c.table[:, 0] = (kind % 3).int()
    c.lens[:] = (kind // 3).int()                       # 0 to 15 rows
    q = torch.randn(48, 2, hd, device="cuda", generator=gen)
    want = c.attention(0, q)
    got = c.attention(0, q[kind], seqs=torch.arange(n, dtype=torch.int32, device="cuda") if listed else None)
    c.sync_status()
    assert torch.equal(got, want[kind])


class Runtime:
    """Captures that torch knows nothing of, through the CUDA runtime that it has loaded."""

    def __init__(self):
        with open("/proc/self/maps") as f:
            paths = {line.split()[-1] for line in f if "libcudart.so" in line}
        if not paths:
            pytest.skip("no shared CUDA runtime")
        self.lib = ctypes.CDLL(sorted(paths)[0])

    def call(self, name, *args):
        assert getattr(self.lib, name)(*args) == 0, name

    def capture(self, stream, work):
        s, graph, run = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
        with torch.cuda.stream(stream):
            self.call("cudaStreamBeginCapture", s, 2)   # (relaxed: allocations are allowed)
            try:
                work()
            finally:
                self.call("cudaStreamEndCapture", s, ctypes.byref(graph))
        self.call("cudaGraphInstantiate", ctypes.byref(run), graph, ctypes.c_ulonglong(0))
        self.call("cudaGraphDestroy", graph)
        return run


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_captures_that_torch_did_not_begin(fmt):
    """Their calls' workspaces stay: memory that is handed out afterwards is not written by a replay."""
    runtime = Runtime()
    c = filled(fmt, 2, 64, 16, [3000, 2500])
    size = c.workspace().numel()
    qs = [torch.randn(2, 4, 64, device="cuda") for _ in range(2)]
    want = [c.attention(0, q).clone() for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        for q, o in zip(qs, outs):
            c.attention(0, q, out=o)

    run = runtime.capture(side, work)
    with torch.cuda.stream(side):
        later = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        runtime.call("cudaGraphLaunch", run, ctypes.c_void_p(side.cuda_stream))
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert all(bool((x == 7).all()) for x in later)
    runtime.call("cudaGraphExecDestroy", run)
    c.sync_status()
    # torch's own captures keep theirs in the graph's pool: nothing more is held here
    held = len(c._captured_workspaces)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    g.replay()
    torch.cuda.synchronize()
    assert held == 2 and len(c._captured_workspaces) == held
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


# ---- the status ---------------------------------------------------------------------

def test_status_of_other_streams_calls_is_not_lost():
    """While a thread reads a status that has a bit of its own, appends on another stream are refused one at a
    time: every refusal is reported by a reading that began before or by the first one that begins after it."""
    c = filled("bf16", 1, 64, 16, [20, 0])
    x = torch.zeros(1, 1, 64, device="cuda")
    bad, at = ints([1]), ints([99])
    side, reader = torch.cuda.Stream(), torch.cuda.Stream()
    rng = np.random.default_rng(0)

    def bits(stream):
        try:
            c.sync_status(stream)
        except dec.DecError as e:
            return ("index" in str(e)) + 2 * ("bad list" in str(e))
        return 0

    for i in range(400):
        torch.cuda.synchronize()
        with torch.cuda.stream(reader):
            c.extend(ints([1, 1]))                      # refused: the reading below has something to clear
        got = []
        t = threading.Thread(target=lambda: got.append(bits(reader)))
        torch.cuda.synchronize()
        torch.cuda._sleep(1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(int(rng.integers(1, 400_000)))  # up to 0.2 ms
            c.append(0, x, x, seqs=bad, positions=at)
        t.start()
        t.join()
        torch.cuda.synchronize()
        got.append(bits(reader))
        assert got[0] & 2 and (got[0] | got[1]) & 1, (i, got)
    c.sync_status()


# ---- pages ------------------------------------------------------------------------

@pytest.mark.parametrize("at", [0, 2, 3, 40])
def test_fork_refuses_pages_that_are_none(at):
    """A parent's entry past the pool, at its first page, further on, its partly filled last one or past it:
    nothing is forked, not even the entry beside it, and the status says so."""
    R, width = 16, 50
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=R, n_pages=12, n_seqs=5, max_pages=width)
    c.extend(ints([0, 1]), ints([3 * R + 5, 20]))
    c.sync_status()
    good = int(c.table[0, at])
    for bad in (12, 1 << 20, 2**31 - 1):
        c.table[0, at] = bad
        state = [t.clone() for t in (c.table, c.lens, c.refs)]
        c.fork(ints([1, 0]), ints([2, 3]))
        with pytest.raises(dec.DecError, match="index"):
            c.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(state, (c.table, c.lens, c.refs)))
    c.table[0, at] = good
    c.fork(ints([1, 0, -1]), ints([2, 3, 4]))
    c.sync_status()
    assert c.lens.tolist() == [3 * R + 5, 20, 20, 3 * R + 5, 0]


def test_fork_of_a_windowed_parent():
    """Entries without a page (freed behind a window) are copied as they are."""
    c = kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, n_pages=12, n_seqs=2, max_pages=8)
    c.extend(ints([0]), ints([100]))
    c.release(ints([0]), window=20, sinks=3)
    c.fork(ints([0]), ints([1]))
    c.sync_status()
    a, b = c.table.cpu().numpy()
    assert list(a >= 0) == list(b >= 0) == [True, False, False, False, False, True, True, False]
    assert list(a == b) == [True, True, True, True, True, True, False, True]
    assert c.refs.cpu().numpy()[a[[0, 5]]].tolist() == [2, 2] and c.refs.cpu().numpy()[[a[6], b[6]]].tolist() == [1, 1]


def test_reads_into_one_tensor_side_by_side():
    """K's rows and V's in turn, or halves of wider rows: taken; the same rows for both: refused."""
    c = filled("q4", 2, 64, 16, [37])
    seqs, pos = ints([0] * 37), ints(range(37))
    want = c.read(0, seqs, pos)
    both = torch.zeros(37, 2, 2, 64, device="cuda")
    c.read(0, seqs, pos, k_out=both[:, 0], v_out=both[:, 1])
    assert torch.equal(both[:, 0], want[0]) and torch.equal(both[:, 1], want[1])
    halves = torch.zeros(2, 37, 2, 64, device="cuda")
    c.read(0, seqs, pos, k_out=halves[1], v_out=halves[0])
    assert torch.equal(halves[1], want[0]) and torch.equal(halves[0], want[1])
    c.sync_status()
    with pytest.raises(dec.DecError, match="overlaps"):
        c.read(0, seqs, pos, k_out=halves[0], v_out=halves[0])
