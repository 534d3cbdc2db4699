"""Rotations by yarn's blend in the pairs' numbers.  Tolerances as in tests/test_gpu_rope.py: 2^-21 of a pair's size,
and half a step of the result's type."""
import numpy as np
import pytest

import kv8_reference as ref
from transformer_layer_decode_gb300 import rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_yarn_by_index(io):
    r = rope.Rotary(128, theta=1e6, scaling="yarn", factor=4.0, context=32768, ramp="index")
    base = rope.Rotary(128, theta=1e6, scaling="yarn", factor=4.0, context=32768)
    x = torch.randn((300, 3, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(io)
    positions = np.arange(300) * 97
    plain = 1e6 ** (-np.arange(64) / 64)
    first, last = 23, 40  # 64 ln(32768 / (2 pi r)) / ln 1e6 is 23.6 for r = 32 and 39.7 for r = 1
    part = np.clip((np.arange(64) - first) / (last - first), 0, 1)
    freq = plain * (1 - part) + plain / 4 * part
    assert np.allclose(r.frequencies, freq, rtol=1e-12) and r.magnitude == base.magnitude
    want = ref.rotate(x.double().cpu().numpy(), positions, freq, np.float64(np.float32(r.magnitude)), "half")
    got = r.rotate(x, torch.tensor(positions, dtype=torch.int32, device="cuda")).double().cpu().numpy()
    size = r.magnitude * (np.abs(x.double().cpu().numpy()) + np.abs(np.roll(x.double().cpu().numpy(), 64, -1)))
    tol = size * 2.0 ** -21 + (np.abs(want) + size * 2.0 ** -21) * torch.finfo(io).eps / 2
    assert (np.abs(got - want) <= tol).all()
