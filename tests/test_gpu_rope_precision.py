"""Rotations to their last bits.

Rows are unit vectors, so a pair's products add an exact 0 and a result is a cosine or a sine.  position * step is
exact modulo whole turns; what is cut off of it, less than 2^-32 turns, is 2 pi * 2^-32 < 0.03 * 2^-24 of an angle.
What rounding the rest to fp32 leaves is made good to its square.  A sine is good to 2 ulp, of 2^-24 at most, and
the FMA that adds that term rounds once more: 2.53 * 2^-24 at most.

The mean tells more.  Two roundings, of the function and of the FMA, each uniform within half a step of the
result (2^-24 in [1/2, 1), which are two thirds of all, less below): sqrt(2 / 12 * (2/3 + 1/3 * 1/5)) = 0.35 * 2^-24 as root
mean square, and a little of the function's own.  Without the term the angle's rounding counts: steps of 2^-24 half
turns for half of all angles, half of that for a quarter, and so on, pi^2 / 12 * (1/2 + 1/16 + 1/128 ..) = 0.47, times
the mean square of a sine, 1/2: with one of the two roundings sqrt(0.235 + 0.061) = 0.54 * 2^-24.  The limit of
0.45 * 2^-24 lies between the two.
"""
import numpy as np
import pytest

from transformer_layer_decode_gb300 import rope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("backward", [False, True])
def test_unit_vectors(layout, backward):
    n, hd = 20000, 64
    rng = np.random.default_rng(4)
    turns = rng.random(hd // 2)                           # of a position; whole turns aside, as steps have it
    freq = turns * 2 * np.pi
    r = rope.Rotary(hd, layout=layout, frequencies=freq)
    positions = rng.integers(0, 1 << 24, n)
    i = np.arange(hd // 2)
    a, b = (i, i + hd // 2) if layout == "half" else (2 * i, 2 * i + 1)
    x = np.zeros((n, 2, hd), np.float32)
    x[:, 0, a] = 1                                        # to (cos, sin)
    x[:, 1, b] = 1                                        # to (-sin, cos)
    y = r.rotate(torch.from_numpy(x).cuda(), torch.tensor(positions, dtype=torch.int32, device="cuda"), backward=backward)
    y = y.double().cpu().numpy()
    # the angle from the steps themselves, whole numbers: exact to 2^-64 turns
    steps = r.steps.cpu().numpy().view(np.uint64)
    with np.errstate(over="ignore"):
        at = (positions.astype(np.uint64)[:, None] * steps).view(np.int64).astype(np.float64) * 2.0 ** -64
    angle = 2 * np.pi * at * (-1 if backward else 1)
    c, s = np.cos(angle), np.sin(angle)
    errors = np.stack([y[:, 0, a] - c, y[:, 0, b] - s, y[:, 1, a] + s, y[:, 1, b] - c]) * 2.0 ** 24
    assert np.abs(errors).max() <= 2.53, np.abs(errors).max()
    assert np.sqrt((errors ** 2).mean()) <= 0.45, np.sqrt((errors ** 2).mean())
