"""CPU checks of how the Python cache makes its calls, with the library's functions replaced."""
import ctypes
import threading
import time

import pytest

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv

MEM = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture
def cache(monkeypatch):
    """A cache without memory or a GPU: what _call needs, on device 0."""
    monkeypatch.setattr(kv, "_current_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 7)
    c = object.__new__(kv.KVCache)
    c._index, c._lock, c.desc = 0, threading.Lock(), kv.KVCacheDesc()
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
