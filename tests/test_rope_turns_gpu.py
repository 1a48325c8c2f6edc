"""Rotary plans: frequencies of the caller's own, and how exact angles are."""
import math

import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

pytestmark = pytest.mark.gpu


def _rotate(rope, positions, x):
    out = torch.empty_like(x, device="cuda")
    ffd.rotate(rope, positions.cuda(), x.cuda(), out)
    return out.cpu().double()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_frequencies_of_the_callers_own(layout):
    """A ramp that runs linearly over the pair index between two pairs, as some models
    have it, written to the plan's turns."""
    d, base, factor, trained, low, high = 128, 10000.0, 8.0, 4096.0, 1.0, 32.0
    rope = ffd.Rope(d, layout, base=base)
    at = [d * math.log(trained / (2 * math.pi * r)) / (2 * math.log(base)) for r in (high, low)]
    f = []
    for i in range(d // 2):
        own = base ** (-2 * i / d)
        g = 1 - min(1.0, max(0.0, (i - at[0]) / (at[1] - at[0])))
        f.append((1 - g) * own / factor + g * own)
        rope.turns[i] = int((f[i] / (2 * math.pi) % 1.0) * 2.0 ** 64)
    x = su.randn(1, 50, 3, 128)
    positions = torch.arange(50, dtype=torch.int32) * 331
    got = _rotate(rope, positions, x)
    want = x.double().clone()
    for i in range(d // 2):
        a, b = (i, i + d // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = (fn(positions.double() * f[i])[:, None] for fn in (torch.cos, torch.sin))
        want[..., a], want[..., b] = x[..., a].double() * c - x[..., b].double() * s, x[..., b].double() * c + x[..., a].double() * s
    assert ((got - want).abs() <= su.rotate_bound(x, want, {})).all()
    # and the plan's own by-parts ramp, linear over the rotations, is another
    other = ffd.Rope(d, layout, base=base, scaling="by_parts", factor=factor, original_length=trained, low=low, high=high)
    assert any(abs(rope.turns[i] - other.turns[i]) > 2 ** 40 for i in range(d // 2))


@pytest.mark.parametrize("position", [1, 12345, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31])
def test_an_angle_is_off_by_2_to_the_minus_26_of_a_turn(position):
    """The pair (1, 0) becomes (cos, sin) of the angle: the plan's fraction times the
    position in whole numbers gives the exact turn.  Off by 2^-26 of a turn moves a
    component by 2 pi 2^-26; cos and sin are fp32 (2^-22 for the function's own error),
    and the result is rounded to bf16."""
    rope = ffd.Rope(128, "interleaved", base=500000.0)
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    x[..., 0::2] = 1.0
    got = _rotate(rope, torch.tensor([position], dtype=torch.int32), x)[0, 0]
    for i in range(64):
        turn = (rope.turns[i] * position) % (1 << 64) / 2.0 ** 64
        for value, want in ((got[2 * i], math.cos(2 * math.pi * turn)), (got[2 * i + 1], math.sin(2 * math.pi * turn))):
            assert abs(float(value) - want) <= abs(want) * 2.0 ** -8 + 2 * math.pi * 2.0 ** -26 + 2.0 ** -22
