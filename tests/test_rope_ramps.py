"""The two ways in which yarn blends kept and divided frequencies (CPU)."""
import ctypes
import math

import numpy as np
import pytest

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec, rope


@pytest.fixture(scope="module")
def lib():
    tld_build.build()
    return dec.load_library()


def frequencies(lib, scaling, rot, theta, factor, context, slow, fast):
    w, m = np.empty(rot // 2), ctypes.c_float()
    rc = lib.dec_rope_frequencies(rot, theta, scaling, factor, context, slow, fast, w.ctypes.data, ctypes.byref(m))
    return rc, w, m.value


def by_index(rot, theta, factor, context, slow, fast):
    """From the definition, pair by pair: the pairs between which the blend runs are found by counting turns."""
    plain = [theta ** (-2 * i / rot) for i in range(rot)]   # (numbers past the last pair count as well)
    turns = [context * w / (2 * math.pi) for w in plain]
    first = max([i for i in range(rot) if turns[i] >= fast], default=0)
    last = min([i for i in range(rot) if turns[i] <= slow], default=rot - 1)
    out = []
    for i, w in enumerate(plain[:rot // 2]):
        part = min(max((i - first) / (last - first), 0), 1) if last > first else float(i > first)
        out.append(w / factor * part + w * (1 - part))
    return np.array(out)


CASES = [(128, 1e4, 8.0, 2048.0, 1.0, 32.0), (128, 1e6, 4.0, 32768.0, 1.0, 32.0), (64, 5e5, 2.5, 8192.0, 1.0, 32.0),
         (96, 1e4, 16.0, 4096.0, 2.0, 8.0), (32, 1e4, 4.0, 100.0, 1.0, 32.0), (128, 1e4, 40.0, 4096.0, 1.0, 32.0),
         (8, 1e4, 4.0, 64.0, 1.0, 1.5), (2, 1e4, 4.0, 64.0, 1.0, 32.0), (64, 10.0, 4.0, 4096.0, 1.0, 32.0)]


@pytest.mark.parametrize("case", CASES)
def test_blend_by_index(lib, case):
    rc, w, m = frequencies(lib, rope.DEC_ROPE_YARN_INDEX, *case)
    assert rc == dec.DEC_OK and m == np.float32(0.1 * math.log(case[2]) + 1)
    assert np.allclose(w, by_index(*case), rtol=1e-12, atol=0)


def test_the_ends_of_a_known_model(lib):
    """128 dimensions, theta 1e4, context 4096: pairs 0 to 20 are kept, those from 46 on divided."""
    _, w, _ = frequencies(lib, rope.DEC_ROPE_YARN_INDEX, 128, 1e4, 16.0, 4096.0, 1.0, 32.0)
    plain = 1e4 ** (-np.arange(64) / 64)
    assert np.allclose(w[:21], plain[:21], rtol=1e-13) and np.allclose(w[46:], plain[46:] / 16, rtol=1e-13)
    assert (w[21:46] < plain[21:46] * (1 - 1e-3)).all() and (w[21:46] > plain[21:46] / 16 * (1 + 1e-3)).all()
    ratio = w / plain
    assert np.allclose(np.diff(ratio[20:47]), -(1 - 1 / 16) / 26, rtol=1e-9)   # a straight line in the pair's number


def test_the_two_differ(lib):
    """As the header says: the same ends, other frequencies between."""
    args = (128, 1e4, 8.0, 2048.0, 1.0, 32.0)
    (_, a, _), (_, b, _) = (frequencies(lib, s, *args) for s in (rope.DEC_ROPE_YARN, rope.DEC_ROPE_YARN_INDEX))
    far = np.maximum(a / b, b / a)
    assert (far > 1.01).sum() == 24 and 2.2 < far.max() < 2.4


@pytest.mark.parametrize("change", [dict(theta=1.0), dict(theta=0.5), dict(context=0.0), dict(context=math.inf), dict(fast=1.0),
                                    dict(slow=-1.0), dict(factor=0.0)])
def test_refusals(lib, change):
    args = dict(rot=64, theta=1e4, factor=4.0, context=2048.0, slow=1.0, fast=32.0)
    assert frequencies(lib, rope.DEC_ROPE_YARN_INDEX, *args.values())[0] == dec.DEC_OK
    args.update(change)
    assert frequencies(lib, rope.DEC_ROPE_YARN_INDEX, *args.values())[0] == dec.DEC_ERR_ARG
    assert frequencies(lib, 5, 64, 1e4, 4.0, 2048.0, 1.0, 32.0)[0] == dec.DEC_ERR_ARG


def test_slow_ends_that_lie_past_the_last_pair(lib):
    rc, w, _ = frequencies(lib, rope.DEC_ROPE_YARN_INDEX, 64, 1e4, 4.0, 1e9, 0.0, 32.0)
    assert rc == dec.DEC_OK and np.isfinite(w).all() and (np.diff(w) < 0).all()


def test_python_says_which():
    for kw in (dict(ramp="line"), dict(ramp="index"), dict(ramp="index", scaling="ntk", factor=2.0),
               dict(ramp="index", frequencies=np.ones(64))):
        with pytest.raises(ValueError, match="ramp"):
            rope.Rotary(128, **kw)
