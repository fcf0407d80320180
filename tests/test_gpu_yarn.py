"""YaRN tables whose ramp ends past the last pair, against the definition written out in 64 bits and
against blends worked out by hand."""

import math

import pytest
import torch

from tests._sana import sana

pytestmark = pytest.mark.gpu


def definition(rot, theta, factor, original, fast, slow):
    """Angle per position of each pair: pairs that turn more than `fast` times over the original
    positions keep their frequency, those that turn less than `slow` times are divided by the factor,
    the rest lies on a straight line over the (whole) pair numbers where they turn that often; these
    are bounded by the rotary elements, 0 to rot - 1."""
    inv = []
    at = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    for j in range(rot // 2):
        f = theta ** (-2 * j / rot)
        g = min(max((j - lo) / (hi - lo if hi > lo else 1e-3), 0.0), 1.0)
        inv.append(f * (1 - g) + f / factor * g)
    return torch.tensor(inv, dtype=torch.float64)


@pytest.mark.parametrize("rot,theta,factor,original,fast,slow", [
    (128, 1e4, 4.0, 131072, 32.0, 1.0),    # ends at pair 70 of 64
    (64, 1e4, 16.0, 1 << 20, 32.0, 1.0),   # 42 of 32
    (32, 1e4, 2.0, 1 << 20, 32.0, 1.0),    # starts at pair 14, ends at 21 of 16
    (16, 100.0, 8.0, 1 << 20, 32.0, 1.0),  # past the rotary elements as well; starts behind the last pair
    (128, 5e5, 8.0, 8192, 32.0, 1.0),      # inside the pairs: as ever
])
def test_tables_follow_the_definition(rot, theta, factor, original, fast, slow):
    n = 4096
    rt = sana.Rotary(n, rot, theta=theta, scaling=("yarn", factor, original, fast, slow, 1.0))
    ang = torch.arange(n, dtype=torch.float64)[:, None] * definition(rot, theta, factor, original, fast, slow)
    t = rt.table.cpu().double()
    # the angle's own rounding in 64 bits (4096 * 2^-50) and one of the result to fp32
    assert (t[..., 0] - torch.cos(ang)).abs().max() <= 2 ** -24
    assert (t[..., 1] - torch.sin(ang)).abs().max() <= 2 ** -24


def test_the_slowest_pair_is_blended():
    """128 elements, theta 1e4, 131072 original positions: pair 63 turns 2.4 times over them, more than
    once, so it is blended and not divided by the whole factor: the ramp runs from pair 45 to 70, and
    18 of its 25 steps lie before pair 63."""
    rt = sana.Rotary(8, 128, scaling=("yarn", 4.0, 131072, 32.0, 1.0, 1.0))
    f = 1e4 ** (-63 / 64)
    assert 131072 * f / (2 * math.pi) > 2.4
    want = f * (1 - 18 / 25) + f / 4 * 18 / 25
    assert abs(rt.table[7, 63, 1].item() - math.sin(7 * want)) <= 2 ** -35  # a step of fp32 at 3.7e-4
