"""CPU checks of 8-bit pages and rotary positions: what is refused before anything is queued, the sizes,
and the frequencies and steps that the host works out."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import kv8_reference as ref
from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, kv, rope

OK, ARG, SHAPE = dec.DEC_OK, dec.DEC_ERR_ARG, dec.DEC_ERR_SHAPE
MEM = 1 << 20  # an aligned address that no call here gets to use


@pytest.fixture(scope="module")
def lib():
    tld_build.build()
    return dec.load_library()


def _cache(**kw):
    base = dict(n_layers=2, n_kv_heads=4, head_dim=128, page_rows=64, n_pages=32, n_seqs=8, max_pages=16,
                format=kv.DEC_KV_Q8T16, pool=MEM, table=MEM, lens=MEM, refs=MEM, status=MEM, scratch=MEM)
    base.update(kw)
    return kv.KVCacheDesc(**base)


def _rope(**kw):
    base = dict(head_dim=128, rot_dim=64, layout=0, magnitude=1.0, steps=MEM)
    base.update(kw)
    return rope.RopeDesc(*base.values())


@pytest.mark.parametrize("hd,R,nkv,layers", [(64, 16, 1, 1), (128, 48, 3, 2), (64, 1024, 1024, 1), (128, 64, 8, 32)])
def test_sizes(lib, hd, R, nkv, layers):
    page, ints, plain = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    c = _cache(head_dim=hd, page_rows=R, n_kv_heads=nkv, n_layers=layers, pool=None)
    assert lib.dec_kv_sizes(ctypes.byref(c), ctypes.byref(page), ctypes.byref(ints)) == OK
    assert page.value == ref.Pages8(nkv, hd, R).page_bytes and page.value % 128 == 0
    c.format = kv.DEC_KV_BF16
    assert lib.dec_kv_sizes(ctypes.byref(c), None, ctypes.byref(plain)) == OK
    assert ints.value == plain.value + layers * 32 * R  # a number for each row of each layer's pages


@pytest.mark.parametrize("kw,code", [({"head_dim": 96}, SHAPE), ({"page_rows": 24}, SHAPE), ({"format": 2}, ARG),
                                     ({"format": 4}, ARG), ({"pool": None}, ARG), ({"pool": MEM + 8}, ARG)])
def test_bad_caches_are_refused(lib, kw, code):
    c, r = ctypes.byref(_cache(**kw)), ctypes.byref(_rope(head_dim=kw.get("head_dim", 128)))
    assert lib.dec_kv_append(c, 0, MEM, MEM, 0, 512, None, None, 1, None) == code
    assert lib.dec_kv_append_rotated(c, 0, r, MEM, MEM, 1024, 1024, 8, MEM, MEM, 0, 512, None, None, 1, None) == code
    assert lib.dec_kv_append_rotated(None, 0, r, MEM, MEM, 1024, 1024, 8, MEM, MEM, 0, 512, None, None, 1, None) == ARG


BAD_ROPES = [({"head_dim": 0}, SHAPE), ({"head_dim": 12, "rot_dim": 4}, SHAPE), ({"head_dim": 1032}, SHAPE),
             ({"rot_dim": 0}, SHAPE), ({"rot_dim": -2}, SHAPE), ({"rot_dim": 7}, SHAPE), ({"rot_dim": 130}, SHAPE),
             ({"layout": 2}, ARG), ({"layout": -1}, ARG), ({"magnitude": math.inf}, ARG), ({"magnitude": math.nan}, ARG),
             ({"steps": None}, ARG), ({"steps": MEM + 4}, ARG)]


@pytest.mark.parametrize("kw,code", BAD_ROPES)
def test_bad_rotations_are_refused(lib, kw, code):
    r, c = ctypes.byref(_rope(**kw)), ctypes.byref(_cache())
    assert lib.dec_rope_rotate(r, MEM, MEM, 0, 1 << 20, 1 << 20, None, 1, 2, 0, None) == code
    assert lib.dec_last_error(None).decode()
    rc = lib.dec_kv_append_rotated(c, 0, r, MEM, MEM, 1024, 1024, 8, MEM, MEM, 0, 512, None, None, 1, None)
    assert rc == code


def test_bad_rotate_calls_are_refused(lib):
    assert lib.dec_rope_rotate(None, MEM, MEM, 0, 256, 256, None, 1, 2, 0, None) == ARG
    r = ctypes.byref(_rope())
    #       x    out      type xs   os   pos  n  heads back
    good = [r, MEM, 2 * MEM, 0, 256, 256, None, 4, 2, 0, None]
    for at, bad, code in ((1, None, ARG), (2, None, ARG), (1, MEM + 4, ARG), (2, MEM + 8, ARG), (3, 2, ARG), (3, -1, ARG),
                          (4, 255, ARG), (4, 258, ARG), (4, -256, ARG), (5, 128, ARG), (5, 257, ARG), (4, (1 << 40) + 4, ARG),
                          (7, -1, ARG), (8, 0, SHAPE), (8, -1, SHAPE), (8, 65537, SHAPE), (7, 1 << 30, SHAPE)):
        args = list(good)
        args[at] = bad
        assert lib.dec_rope_rotate(*args) == code, (at, bad)
    args = list(good)
    args[2], args[4], args[5] = MEM, 256, 512            # in place with other strides
    assert lib.dec_rope_rotate(*args) == ARG
    args = list(good)
    args[2] = MEM + 1024 * 4 - 16                        # out begins in x's last bytes
    assert lib.dec_rope_rotate(*args) == ARG
    args = list(good)
    args[7], args[1] = 0, None
    assert lib.dec_rope_rotate(*args) == OK              # nothing to do


def test_bad_rotated_appends_are_refused(lib):
    c, r = ctypes.byref(_cache()), ctypes.byref(_rope())
    #       0  1  2  q    q_out    qs    qos   heads k        v        type stride seqs positions n
    good = [c, 1, r, MEM, 2 * MEM, 1024, 1024, 8, 3 * MEM, 4 * MEM, 0, 512, None, None, 2, None]
    for at, bad, code in ((1, 2, ARG), (1, -1, ARG), (2, None, ARG), (3, None, ARG), (4, None, ARG), (4, MEM + 16, ARG),
                          (5, 1023, ARG), (6, 1000, ARG), (5, 1025, ARG), (7, -1, SHAPE), (7, 65537, SHAPE), (8, None, ARG),
                          (9, None, ARG), (8, MEM + 4, ARG), (10, 2, ARG), (11, 511, ARG), (11, 513, ARG), (14, -1, ARG),
                          (14, 9, ARG)):
        args = list(good)
        args[at] = bad
        assert lib.dec_kv_append_rotated(*args) == code, (at, bad)
    r64 = ctypes.byref(_rope(head_dim=64))
    assert lib.dec_kv_append_rotated(c, 1, r64, *good[3:]) == SHAPE
    # q_out over k: in the same wide rows as it, and between them
    args = list(good)
    args[4], args[6], args[11], args[14] = 3 * MEM + 512 * 4 - 16, 2048, 2048, 2
    assert lib.dec_kv_append_rotated(*args) == ARG
    args[4], args[8] = 3 * MEM, 3 * MEM + (2048 - 500) * 4
    assert lib.dec_kv_append_rotated(*args) == ARG
    args = list(good)
    args[14] = 0
    assert lib.dec_kv_append_rotated(*args) == OK


@pytest.mark.parametrize("n,wa,wb,at,overlap", [  # rows 100 apart; b begins `at` behind a
    (3, 60, 40, 60, False), (3, 60, 40, 59, True), (3, 60, 41, 60, True), (1, 60, 40, 60, False), (1, 60, 41, 60, False),
    (3, 60, 40, -40, False), (3, 60, 41, -40, True), (3, 60, 40, 0, True), (3, 10, 10, 300, False), (3, 10, 10, 200, True)])
def test_rows_of_one_wide_tensor(tmp_path, n, wa, wb, at, overlap):
    """The q, k and v of one projection's rows lie beside each other: that is no overlap."""
    import os
    import subprocess
    here = os.path.dirname(os.path.abspath(__file__))
    src = tmp_path / "overlap.cpp"
    src.write_text('#include "kv.h"\nint main() { return tld::kv_rows_overlap(10000, 100, %d, 10000 + (%d), 100, %d, %d); }\n'
                   % (wa, at, wb, n))
    csrc = os.path.join(os.path.dirname(here), "transformer_layer_decode_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, "-I/usr/local/cuda/include", str(src), "-o", str(tmp_path / "x")],
                   check=True)
    brute = any(10000 + 100 * i < 10000 + at + 100 * j + wb and 10000 + at + 100 * j < 10000 + 100 * i + wa
                for i in range(n) for j in range(n))
    assert brute == overlap and subprocess.run([str(tmp_path / "x")]).returncode == int(overlap)


@pytest.mark.parametrize("rot", [2, 4, 64, 100, 128])
@pytest.mark.parametrize("name,kw", [(None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                     ("yarn", dict(factor=8.0, context=4096.0)),
                                     ("yarn", dict(factor=2.5, context=8192.0, slow=1.0, fast=4.0))])
def test_frequencies(lib, rot, name, kw):
    w, m = np.empty(rot // 2), ctypes.c_float()
    a = dict(theta=5e5, factor=1.0, context=0.0, slow=1.0, fast=32.0)
    a.update(kw)
    rc = lib.dec_rope_frequencies(rot, a["theta"], rope.SCALINGS[name], a["factor"], a["context"], a["slow"], a["fast"],
                                  w.ctypes.data, ctypes.byref(m))
    if name == "ntk" and rot == 2:
        assert rc == SHAPE
        return
    assert rc == OK
    want, magnitude = ref.frequencies(rot, scaling=name, **a)
    assert np.allclose(w, want, rtol=1e-14, atol=0) and m.value == np.float32(magnitude)
    if name == "ntk" and rot > 2:  # the fastest stays, the slowest is divided by the factor
        plain, _ = ref.frequencies(rot, theta=5e5)
        assert np.isclose(w[0], plain[0]) and np.isclose(w[-1], plain[-1] / a["factor"])


@pytest.mark.parametrize("args", [(0, 1e4, 0, 1, 0, 1, 32), (3, 1e4, 0, 1, 0, 1, 32), (1026, 1e4, 0, 1, 0, 1, 32),
                                  (64, 0.0, 0, 1, 0, 1, 32), (64, math.inf, 0, 1, 0, 1, 32), (64, math.nan, 0, 1, 0, 1, 32),
                                  (64, 1e4, 4, 1, 0, 1, 32), (64, 1e4, -1, 1, 0, 1, 32), (64, 1e4, 1, 0.0, 0, 1, 32),
                                  (64, 1e4, 2, -1.0, 0, 1, 32), (64, 1e4, 3, 2, 0, 1, 32), (64, 1e4, 3, 2, 2048, 8, 8),
                                  (64, 1e4, 3, 2, 2048, -1, 8)])
def test_bad_frequencies_are_refused(lib, args):
    w = np.empty(1024)
    assert lib.dec_rope_frequencies(*args, w.ctypes.data, None) in (ARG, SHAPE)
    assert lib.dec_rope_frequencies(64, 1e4, 0, 1, 0, 1, 32, None, None) == ARG


def test_steps(lib):
    """Within 2^-64 of a turn (and what 2 pi's two doubles leave of a large frequency), whole turns aside."""
    pi = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    f = np.array([1.0, 1e4 ** -0.5, 5e5 ** (-126 / 128), 0.0, -1.0, 2 * math.pi, 100.0, -1e-12, 1e-18, 1e6, -1e6])
    steps = np.empty(len(f), np.uint64)
    assert lib.dec_rope_steps(f.ctypes.data, len(f), steps.ctypes.data) == OK
    for x, got in zip(f, steps):
        want = Fraction(float(x)) / (2 * pi) * 2 ** 64
        off = (Fraction(int(got)) - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= 2 + abs(want) / 2 ** 96, (x, float(off))
    for bad in (math.nan, math.inf, 2e6):
        assert lib.dec_rope_steps(np.array([bad]).ctypes.data, 1, steps.ctypes.data) == ARG
    assert lib.dec_rope_steps(None, 1, steps.ctypes.data) == ARG
    assert lib.dec_rope_steps(None, 0, None) == OK


def test_python_refuses_before_it_calls():
    for kw, word in (({"layout": "halves"}, "layout"), ({"scaling": "cubic"}, "scaling"), ({"rot_dim": 130}, "rot_dim"),
                     ({"rot_dim": 3}, "rot_dim"), ({"rot_dim": 1 << 33}, "rot_dim"), ({"frequencies": [1.0]}, "frequencies"),
                     ({"frequencies": np.ones(64), "scaling": "linear"}, "not scaled"), ({"magnitude": math.nan}, "magnitude"),
                     ({"device": "cpu"}, "CUDA")):
        with pytest.raises(ValueError, match=word):
            rope.Rotary(128, **kw)
    for hd in (0, 12, 1032, (1 << 32) + 64):
        with pytest.raises(ValueError, match="head_dim"):
            rope.Rotary(hd)
    with pytest.raises(dec.DecError, match="factor"):
        rope.Rotary(128, scaling="linear", factor=0.0)


def test_reference_blocks():
    """The statement of a block's writing: a value is off by half a step, and by one after any number of growths."""
    rng = np.random.default_rng(2)
    p = ref.Pages8(2, 64, 32)
    page = rng.integers(0, 256, p.page_bytes).astype(np.uint8)
    rows = {}
    for r in range(16):                                  # one at a time, ever larger
        x = (rng.normal(0, 1, (2, 2, 64)) * 1.5 ** r).astype(np.float32)
        p.write(page, 1, {r: x})
        rows[r] = x
    v, s = p.values(page)[:, :, 16:], p.parts(page)[1]
    for r, x in rows.items():
        assert np.all(np.abs(v[:, :, r] - x) <= np.stack([a[:, 1] for a in s])[..., None])
    p.write(page, 1, {0: rows[0], 5: rows[5]})           # from the first row on: nothing of before
    v, s = p.values(page)[:, :, 16:], p.parts(page)[1]
    for i in range(2):
        for h in range(2):
            top = max(np.abs(rows[0][i, h]).max(), np.abs(rows[5][i, h]).max())
            step = s[i][h, 1]
            assert top <= 127 * step and (top > 127 * step / 2) and math.frexp(step)[0] == 0.5
            assert np.all(np.abs(v[i, h, 5] - rows[5][i, h]) <= step / 2)
    assert ref.scale_exponent(127.0) == 0 and ref.scale_exponent(np.nextafter(127.0, 128.0)) == 1
    assert ref.scale_exponent(3.4e38) == 121 and ref.scale_exponent(1e-45) == -126
