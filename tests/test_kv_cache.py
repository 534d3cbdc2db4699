"""CPU checks of the paged cache's calls: what is refused before anything is
queued, the sizes, and the plain statements its GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import kv_reference as ref
from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv

OK, ARG, SHAPE = dec.DEC_OK, dec.DEC_ERR_ARG, dec.DEC_ERR_SHAPE
MEM = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture(scope="module")
def lib():
    tld_build.build()
    return dec.load_library()


def _desc(**kw):
    base = dict(n_layers=2, n_kv_heads=4, head_dim=128, page_rows=64, n_pages=32, n_seqs=8, max_pages=16,
                format=0, pool=MEM, table=MEM, lens=MEM, refs=MEM, status=MEM, scratch=MEM)
    base.update(kw)
    return kv.KVCacheDesc(**base)


@pytest.mark.parametrize("kw,code", [
    ({"head_dim": 96}, SHAPE), ({"head_dim": 0}, SHAPE), ({"page_rows": 0}, SHAPE), ({"page_rows": 24}, SHAPE),
    ({"page_rows": 1040}, SHAPE), ({"n_layers": 0}, SHAPE), ({"n_kv_heads": 0}, SHAPE), ({"n_kv_heads": -1}, SHAPE),
    ({"n_pages": 0}, SHAPE), ({"n_pages": (1 << 20) + 1}, SHAPE), ({"n_seqs": 0}, SHAPE), ({"n_seqs": 65537}, SHAPE),
    ({"max_pages": 0}, SHAPE), ({"max_pages": 1 << 30}, SHAPE), ({"format": 2}, ARG), ({"format": -1}, ARG),
])
def test_bad_shapes_are_refused_by_every_call(lib, kw, code):
    c = ctypes.byref(_desc(**kw))
    n = ctypes.c_size_t()
    assert lib.dec_kv_sizes(c, ctypes.byref(n), None) == code
    assert lib.dec_last_error(None).decode()
    assert lib.dec_kv_append(c, 0, MEM, MEM, 0, 512, None, None, 1, None) == code
    assert lib.dec_kv_read(c, 0, MEM, MEM, 0, 512, None, None, 1, None) == code
    assert lib.dec_kv_attention(c, 0, MEM, 2 * MEM, 0, 1024, 1024, None, 1, 8, 0, 0, 0.0, MEM, 1 << 40, None) == code
    assert lib.dec_kv_attention_workspace(c, ctypes.byref(n)) == code
    assert lib.dec_kv_extend(c, None, None, 1, None) == code
    assert lib.dec_kv_fork(c, MEM, MEM, 1, None) == code
    assert lib.dec_kv_release(c, None, 1, 0, 0, None) == code
    assert lib.dec_kv_compact(c, None) == code
    assert lib.dec_kv_status(c, None, None) == code


@pytest.mark.parametrize("kw", [{p: None} for p in ("pool", "table", "lens", "refs", "status", "scratch")]
                         + [{"pool": MEM + 8}, {"table": MEM + 2}, {"scratch": MEM + 1}])
def test_bad_memory_is_refused(lib, kw):
    c = ctypes.byref(_desc(**kw))
    assert lib.dec_kv_sizes(c, None, None) == OK  # looks at no pointer
    assert lib.dec_kv_append(c, 0, MEM, MEM, 0, 512, None, None, 1, None) == ARG
    assert lib.dec_kv_attention(c, 0, MEM, 2 * MEM, 0, 1024, 1024, None, 1, 8, 0, 0, 0.0, MEM, 1 << 40, None) == ARG
    assert lib.dec_kv_extend(c, None, None, 1, None) == ARG
    assert lib.dec_kv_compact(c, None) == ARG
    assert lib.dec_kv_status(c, None, None) == ARG


def test_null_cache_is_an_error(lib):
    assert lib.dec_kv_sizes(None, None, None) == ARG
    assert lib.dec_kv_append(None, 0, MEM, MEM, 0, 512, None, None, 1, None) == ARG
    assert lib.dec_kv_attention(None, 0, MEM, MEM, 0, 1024, 1024, None, 1, 8, 0, 0, 0.0, MEM, 64, None) == ARG
    assert lib.dec_kv_compact(None, None) == ARG


def test_bad_rows_calls_are_refused(lib):
    c = ctypes.byref(_desc())
    for fn in (lib.dec_kv_append, lib.dec_kv_read):
        good = [c, 1, MEM, MEM, 0, 512, None, None, 1, None]
        for at, bad in ((1, -1), (1, 2), (2, None), (3, None), (4, 2), (4, -1), (5, 511), (5, 0), (5, -512), (5, 513),
                        (2, MEM + 4), (3, MEM + 8), (8, -1), (8, 9)):
            args = list(good)
            args[at] = bad
            assert fn(*args) == ARG, (at, bad)
        args = list(good)
        args[8] = 0
        assert fn(*args) == OK                     # nothing to do
        args[2] = None
        assert fn(*args) == OK
    # bf16 rows: 8 elements are 16 bytes
    assert lib.dec_kv_append(c, 0, MEM, MEM, 1, 516, None, None, 1, None) == ARG


def test_bad_attention_calls_are_refused(lib):
    c = ctypes.byref(_desc())
    #        layer q    o        type qs    os    seqs n  nq win sinks scale ws   bytes
    good = [c, 1, MEM, 2 * MEM, 0, 1024, 1024, None, 1, 8, 0, 0, 0.0, MEM, 1 << 40, None]
    for at, bad in ((1, -1), (1, 2), (2, None), (3, None), (2, MEM + 4), (3, MEM + 4), (4, 2), (5, 1023), (5, 1025),
                    (6, 1000), (6, -1024), (8, -1), (8, 9), (8, 65536), (10, -1), (11, -1), (12, float("nan")),
                    (12, float("inf")), (13, None), (13, MEM + 8), (14, 0)):
        args = list(good)
        args[at] = bad
        rc = lib.dec_kv_attention(*args)
        # (without a GPU the size that a workspace must have may not be known)
        assert rc == ARG or (at in (13, 14) and rc == dec.DEC_ERR_CUDA), (at, bad, rc)
    for heads in (0, -4, 6, 9):
        args = list(good)
        args[9] = heads
        assert lib.dec_kv_attention(*args) == SHAPE
    args = list(good)
    args[3] = MEM                                        # o = q
    assert lib.dec_kv_attention(*args) == ARG
    args[3] = MEM + 1024 * 4 - 16                        # o begins in q's last bytes
    assert lib.dec_kv_attention(*args) == ARG
    args = list(good)
    args[7], args[8], args[5], args[6] = MEM, 4, 4096, 4096
    args[3] = MEM + 512 * 4                              # q and o share half of each of the same wide rows
    assert lib.dec_kv_attention(*args) == ARG
    args = list(good)
    args[8] = 0
    assert lib.dec_kv_attention(*args) == OK
    n = ctypes.c_size_t()
    assert lib.dec_kv_attention_workspace(c, None) == ARG


def test_bad_page_calls_are_refused(lib):
    c = ctypes.byref(_desc())
    for n in (-1, 9):
        assert lib.dec_kv_extend(c, MEM, MEM, n, None) == ARG
        assert lib.dec_kv_fork(c, MEM, MEM, n, None) == ARG
        assert lib.dec_kv_release(c, MEM, n, 0, 0, None) == ARG
    assert lib.dec_kv_fork(c, None, MEM, 1, None) == ARG
    assert lib.dec_kv_fork(c, MEM, None, 1, None) == ARG
    assert lib.dec_kv_release(c, MEM, 1, -1, 0, None) == ARG
    assert lib.dec_kv_release(c, MEM, 1, 4, -1, None) == ARG
    assert lib.dec_kv_extend(c, None, None, 0, None) == OK
    assert lib.dec_kv_fork(c, None, None, 0, None) == OK
    assert lib.dec_kv_release(c, None, 0, 0, 0, None) == OK


@pytest.mark.parametrize("fmt,hd,R,nkv", [(0, 64, 128, 2), (0, 128, 16, 3), (1, 64, 16, 1), (1, 128, 1024, 8)])
def test_sizes(lib, fmt, hd, R, nkv):
    page, ints = ctypes.c_size_t(), ctypes.c_size_t()
    c = _desc(format=fmt, head_dim=hd, page_rows=R, n_kv_heads=nkv, pool=None)
    assert lib.dec_kv_sizes(ctypes.byref(c), ctypes.byref(page), ctypes.byref(ints)) == OK
    assert page.value == ref.Pages("q4" if fmt else "bf16", nkv, hd, R).page_bytes
    assert page.value % 16 == 0 and ints.value >= 2 * 32 + 3 * 8


def test_python_refuses_before_it_calls():
    with pytest.raises(ValueError, match="fmt"):
        kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, n_pages=1, n_seqs=1, max_pages=1, fmt="int8")
    with pytest.raises(ValueError, match="needed"):
        kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, n_pages=1)
    with pytest.raises(ValueError, match="together"):
        kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=64, pool=np.zeros(4))
    with pytest.raises(dec.DecError):
        kv.KVCache(n_layers=1, n_kv_heads=1, head_dim=80, n_pages=1, n_seqs=1, max_pages=1)


def test_reference_rows_round_trip():
    """The layout's two directions agree, and the codes are the nearest ones."""
    rng = np.random.default_rng(3)
    for hd in (64, 128):
        p = ref.Pages("q4", 2, hd, 16)
        page = rng.integers(0, 256, p.page_bytes).astype(np.uint8)
        rows = {}
        for which in range(2):
            for head in range(2):
                for row in range(16):
                    x = rng.normal(0, 1, hd).astype(np.float32)
                    p.put(page, which, head, row, x)
                    rows[which, head, row] = x
        vals = p.values(page)
        for (w, h, r), x in rows.items():
            c, s = ref.q4_encode(x)
            assert np.array_equal(vals[w, h, r], ref.q4_value(c, s))
            # nearest: within half a step, and the scale's own rounding at the ends (7.5 of 7.004 steps)
            assert np.all(np.abs(vals[w, h, r] - x) <= 0.5001 * np.repeat(s.astype(np.float64), 32))


def test_reference_model_counts_pages():
    """A walk of the page model leaves no page lost: refs are what the tables name."""
    rng = np.random.default_rng(5)
    m = ref.Model(40, 10, 12, 16)
    for _ in range(400):
        op = rng.integers(0, 5)
        if op == 0:
            m.extend(rng.permutation(10)[:3], rng.integers(0, 40, 3))
        elif op == 1:
            m.fork(rng.integers(0, 10, 2), rng.permutation(10)[:2])
        elif op == 2:
            m.release(rng.integers(-1, 10, 2))
        elif op == 3:
            m.release(range(10), window=30, sinks=4)
        else:
            m.compact()
        named = np.bincount(m.table[m.table >= 0], minlength=40)
        assert np.array_equal(named, m.refs)
    assert m.bits


def test_codes_without_divisions(tmp_path):
    """The quotients behind the 4-bit codes and scales, against IEEE division and 64 bits."""
    exe = tmp_path / "kv_codes_check"
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host", "kv_codes_check.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", src, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout
