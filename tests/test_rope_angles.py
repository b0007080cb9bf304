"""Angles of the rotation against decimal arithmetic of 60 digits: good to 2^-25 of a turn and 2^-50 of the angle,
for any position and base. The outputs here are the cosine and the sine themselves (rotation of (1, 0) without
a norm): 2 steps each, 4 U, on top."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

import adaln_layernorm_modulate_gb300 as A

U = 2.0 ** -24
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
POSITIONS = [0, 1, -1, 2, 3, 17, 4096, 32759, 500000, -500001, 2 ** 24 + 1, 1234567891, -987654321, 2 ** 31 - 1,
             -(2 ** 31)]


def turns(theta, w, pos):
    """[positions][pairs]: (fraction of a turn in [-1/2, 1/2], the angle's size in radians)."""
    getcontext().prec = 60
    out = []
    for p in pos:
        row = []
        for i in range(w // 2):
            t = p * Decimal(theta) ** (Decimal(-2 * i) / w) / (2 * PI)
            row.append((float(t - t.to_integral_value()), abs(float(t * 2 * PI))))
        out.append(row)
    return out


def test_the_decimal_turns():
    for theta, w in ((10000.0, 16), (1.0, 8), (1e12, 24)):
        for p, row in zip((0, 3, -40), turns(theta, w, (0, 3, -40))):
            for i, (t, size) in enumerate(row):
                angle = p * theta ** (-2.0 * i / w)
                assert abs(size - abs(angle)) <= 1e-14 * size
                assert abs(math.cos(2 * math.pi * t) - math.cos(angle)) <= 1e-13
                assert abs(math.sin(2 * math.pi * t) - math.sin(angle)) <= 1e-13


@pytest.mark.gpu
@pytest.mark.parametrize("theta", [1.0, 10000.0, 500000.0, 1e12, 1e300])
@pytest.mark.parametrize("w", [2, 42, 64, 128])
def test_angles(theta, w):
    ref = torch.tensor(turns(theta, w, POSITIONS), dtype=torch.float64, device="cuda")
    R = len(POSITIONS)
    pos = torch.tensor(POSITIONS, dtype=torch.int64).to(torch.int32).cuda()[:, None]
    x = torch.zeros(R, w, device="cuda")
    x[:, 0::2] = 1
    d = (w + 7) // 8 * 8
    q = torch.nn.functional.pad(x, (0, d - w)).contiguous()
    out = torch.empty_like(q)
    A.adaln_qk_norm_rope_fwd(q, None, None, None, pos, out, None, R, 1, 0, d, d, 0, d, 0, (w,), theta, norm=False)
    angle = 2 * math.pi * ref[..., 0]
    err = 2 * math.pi * 2.0 ** -25 + ref[..., 1] * 2.0 ** -50 + 4 * U
    assert ((out[:, 0:w:2].double() - angle.cos()).abs() <= err).all()
    assert ((out[:, 1:w:2].double() - angle.sin()).abs() <= err).all()
