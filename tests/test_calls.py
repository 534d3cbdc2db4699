"""The module that marshals a decode step's calls: what it does not know to be right it leaves to Python's checks."""
import ctypes

import pytest
import torch

from transformer_layer_decode_gb300 import build as tld_build
from transformer_layer_decode_gb300 import dec

CALLED = []
CALL = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: CALLED.append(1) or 0)


@pytest.fixture(scope="module")
def fast():
    tld_build.build()
    return dec.load_calls()


def test_tensors_elsewhere_are_left_to_python(fast):
    f = ctypes.cast(CALL, ctypes.c_void_p).value
    c = fast.context(1 << 20, 0, 4, 128, f, f, f, f)
    r = fast.context(1 << 20, 0, 0, 128, f)
    k, seqs = torch.zeros(2, 4, 128), torch.zeros(2, dtype=torch.int32)
    for x in (k, k.half(), k[0], None, 3, "k", k.numpy()):
        assert fast.append(c, 0, x, x, None, None) is None
        assert fast.read(c, 0, x, x, seqs, None) is None
        assert fast.append_rotated(c, 0, x, x, None, None, r, None, None) is None
        assert fast.attention(c, 0, x, x, None, 0, 0, 0.0, 1 << 20, 1 << 20) is None
        assert fast.rotate(r, x, seqs, x, False) is None
    assert fast.append_rotated(c, 0, k, k, None, None, None, None, None) is None
    assert not CALLED


def test_misuse_is_an_error(fast):
    c = fast.context(1 << 20, 0, 4, 128, 0)
    for f in (fast.append, fast.read, fast.append_rotated, fast.attention, fast.rotate):
        with pytest.raises(TypeError):
            f(c)
    with pytest.raises(ValueError):
        fast.rotate(3, None, None, None, False)
    with pytest.raises(TypeError):
        fast.context("here", 0, 4, 128, 0)
