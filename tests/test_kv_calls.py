"""CPU checks of how the Python cache makes its calls, with the library's functions replaced."""
import ctypes
import threading
import time

import pytest
import torch

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv

MEM = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture
def cache(monkeypatch):
    """A cache without memory or a GPU: what _call needs, on device 0."""
    monkeypatch.setattr(kv, "_current_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 7)
    c = object.__new__(kv.KVCache)
    c._index, c._lock, c._status_lock, c.desc = 0, threading.Lock(), threading.Lock(), kv.KVCacheDesc()
    c._ref = ctypes.byref(c.desc)
    return c


def test_calls_of_two_threads_do_not_interleave(cache):
    """A call is several launches: while one is being queued no other thread's is."""
    inside, seen = [], []

    def call(ref, who, stream):
        inside.append(who)
        time.sleep(0.002)           # another thread gets to run, as it does while the library's function runs
        seen.append(list(inside))
        inside.remove(who)
        return 0

    def work(who):
        for _ in range(10):
            cache._call(call, who)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 30 and all(len(s) == 1 for s in seen)


def test_a_reading_of_the_status_holds_no_other_call_up(cache):
    """It waits for its stream: what other threads queue meanwhile goes ahead, but for other readings."""
    go, order = threading.Event(), []

    class Lib:
        @staticmethod
        def dec_kv_status(ref, bits, stream):
            order.append("waits")
            assert go.wait(20)
            order.append("has waited")
            return 0

    cache.lib = Lib
    readers = [threading.Thread(target=cache.sync_status) for _ in range(2)]
    for t in readers:
        t.start()
    try:
        other = threading.Thread(target=cache._call, args=(lambda ref, stream: 0,))
        other.start()
        other.join(10)
        assert not other.is_alive() and all(t.is_alive() for t in readers)
    finally:
        go.set()
        for t in readers:
            t.join()
    assert order == ["waits", "has waited"] * 2


@pytest.mark.parametrize("handle,shared", [(7, True), (2, False)])
def test_streams_that_are_each_thread_s_own_share_no_workspace(cache, monkeypatch, handle, shared):
    """Calls of one stream run one after another and share a workspace; the handle of the per-thread default
    stream names as many streams as there are threads."""
    monkeypatch.setattr(kv, "_raw_stream", lambda index: handle)
    monkeypatch.setattr(kv, "_capturing", lambda: False)
    cache.device, cache._d, cache._workspaces = torch.device("cpu"), 64, {}
    cache.lib = type("Lib", (), {"dec_kv_attention": None})
    monkeypatch.setattr(kv.KVCache, "workspace", lambda self: torch.empty(16, dtype=torch.uint8))
    used = {}
    monkeypatch.setattr(kv.KVCache, "_call", lambda self, fn, *args, stream=None: used.setdefault(
        threading.get_ident(), []).append(args[-2]))
    both = threading.Barrier(2)

    def work(turn):
        if turn:
            both.wait(10)
        for _ in range(2):
            cache.attention(0, torch.zeros(1, 2, 64))
        if not turn:
            both.wait(10)
        both.wait(10)               # (both threads live as long as the other's calls)

    threads = [threading.Thread(target=work, args=(turn,)) for turn in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    a, b = used.values()
    assert a[0] == a[1] and b[0] == b[1] and (a[0] == b[0]) == shared


@pytest.fixture(scope="module")
def lib():
    tld_build.build()
    return dec.load_library()


@pytest.mark.parametrize("n,heads,code", [
    (65536, 1, dec.DEC_ERR_CUDA), (65536, 256, dec.DEC_ERR_CUDA), (256, 65536, dec.DEC_ERR_CUDA),
    (65537, 1, dec.DEC_ERR_ARG), (65536, 257, dec.DEC_ERR_SHAPE), (1, 65537, dec.DEC_ERR_SHAPE)])
def test_the_most_queries_and_heads(lib, n, heads, code):
    """What the header allows gets as far as the device, which is not there; one more does not."""
    # a workspace at no multiple of 16: refused after the sizes, should there be a device
    c = kv.KVCacheDesc(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, n_pages=32, n_seqs=65536, max_pages=1, format=0,
                       pool=MEM, table=MEM, lens=MEM, refs=MEM, status=MEM, scratch=MEM)
    width = 64 * heads
    for seqs in (None, MEM):
        rc = lib.dec_kv_attention(ctypes.byref(c), 0, MEM, 1 << 50, 0, width, width, seqs, n, heads, 0, 0, 0.0, MEM + 4,
                                  1 << 40, None)
        if code == dec.DEC_ERR_CUDA and rc == dec.DEC_ERR_ARG:
            assert "workspace" in dec.load_library().dec_last_error(None).decode()
        else:
            assert rc == code


@pytest.mark.parametrize("kw", [
    {"n_layers": 2**32 + 1}, {"n_kv_heads": 2**32 + 2}, {"head_dim": 2**32 + 64}, {"page_rows": 2**32 + 16},
    {"n_pages": 2**32 + 4}, {"n_seqs": -2**32 + 2}, {"max_pages": 2**32 + 1}])
def test_shapes_past_32_bits_are_refused(kw):
    """Not cut off to a shape that is allowed."""
    shape = dict(n_layers=1, n_kv_heads=2, head_dim=64, page_rows=16, n_pages=4, n_seqs=2, max_pages=1)
    shape.update(kw)
    with pytest.raises(ValueError, match=next(iter(kw))):
        kv.KVCache(**shape)


def test_arguments_past_32_bits_are_refused(cache, monkeypatch):
    monkeypatch.setattr(kv, "_capturing", lambda: False)
    cache.device, cache._d, cache.lib = torch.device("cpu"), 64, dec.load_library()
    cache.desc.n_kv_heads, cache.desc.n_layers, cache.desc.n_seqs = 2, 3, 2
    called = []
    monkeypatch.setattr(kv.KVCache, "_call", lambda self, fn, *args, stream=None: called.append(args))
    x, ws, list_ = torch.zeros(2, 2, 64), torch.zeros(64), torch.zeros(2, dtype=torch.int32)

    def attend(**kw):
        cache.attention(kw.pop("layer", 1), x, out=torch.zeros(2, 2, 64), workspace=ws, **kw)

    for big in (2**32, 2**32 + 1, 2**31, -2**31 - 1, -2**32):
        for name in ("layer", "window", "sinks"):
            with pytest.raises(ValueError, match=name):
                attend(**{name: big})
        with pytest.raises(ValueError, match="layer"):
            cache.append(big, x, x)
        with pytest.raises(ValueError, match="layer"):
            cache.read(big, list_, k_out=x, v_out=x)
        for name in ("window", "sinks"):
            with pytest.raises(ValueError, match=name):
                cache.release(**{name: big})
    assert not called
    attend(window=2**31 - 1, sinks=2**31 - 1)
    attend(window=-1)                    # (the library's to refuse)
    cache.release(window=5, sinks=-2)
    assert len(called) == 3


def test_scales_past_fp32_are_refused(lib):
    """The kernels take the scale times log2(e)."""
    c = kv.KVCacheDesc(n_layers=1, n_kv_heads=1, head_dim=64, page_rows=16, n_pages=32, n_seqs=8, max_pages=1, format=0,
                       pool=MEM, table=MEM, lens=MEM, refs=MEM, status=MEM, scratch=MEM)

    def rc(scale, n=0):
        return lib.dec_kv_attention(ctypes.byref(c), 0, MEM, 2 * MEM, 0, 64, 64, None, n, 1, 0, 0, scale, MEM, 1 << 40, None)

    for scale in (3e38, -2.4e38, float("inf"), float("-inf"), float("nan"), 1e300):
        assert rc(scale) == rc(scale, 1) == dec.DEC_ERR_ARG
    for scale in (0.0, -0.0, 2.3e38, -1.0, 1e-45):
        assert rc(scale) == dec.DEC_OK


def test_reads_into_rows_that_overlap_are_refused(lib):
    """K's rows and V's, of 512 bytes here, would be written in any order."""
    c = kv.KVCacheDesc(n_layers=1, n_kv_heads=2, head_dim=64, page_rows=16, n_pages=32, n_seqs=8, max_pages=1, format=0,
                       pool=MEM, table=MEM, lens=MEM, refs=MEM, status=MEM, scratch=MEM)

    def rc(v, stride, n):
        lib.dec_kv_sizes(None, None, None)   # (some other message)
        rc = lib.dec_kv_read(ctypes.byref(c), 0, MEM, v, 0, stride, MEM, None, n, None)
        return rc, "overlaps" in lib.dec_last_error(None).decode()

    for v, stride, n in ((MEM, 128, 1), (MEM + 496, 128, 1), (MEM + 512, 128, 2), (MEM + 256, 256, 2), (MEM - 16, 256, 2),
                         (MEM + 1024, 128, 100), (MEM + 3 * 1024 + 400, 256, 9)):
        assert rc(v, stride, n) == (dec.DEC_ERR_ARG, True), (v - MEM, stride, n)
        assert rc(v, stride, 0) == (dec.DEC_OK, False)
