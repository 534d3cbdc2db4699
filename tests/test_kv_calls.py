"""CPU checks of how the Python cache makes its calls, with the library's functions replaced."""
import ctypes
import threading
import time

import pytest

from transformer_layer_decode_gb300 import kv


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
