"""Angles of the rotary store at far positions, where a rotation by nearly a quarter turn
leaves little: what is left shows the angle's error.

With x = 1 and y = 0 the pair becomes (cos phi, sin phi).  The frequency is a double, and its
turns per position are taken to 2^-65, so the fraction of a turn is off by pos 2^-65 (2^-34);
its upper 32 bits are kept (2^-32) and become an fp32 number of half turns up to 1 (2^-25, that
is 2^-26 turns); an angle error moves cos and sin by 2 pi as much at most.  sincospi is off by
2 units in the last place (2^-22 of the value), the value rounds to bf16 (2^-8)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_step_ops_gpu import _built, i32  # noqa: F401

pytestmark = pytest.mark.gpu

FREQ = [6.0, 5.9, 4.7123, 3.3333, 2.0 + 2.0 ** -51, 1.0, 0.123456789, 1e-3]
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)


def turns(f, bits):
    """f / 2 pi in units of 2^-bits, as an integer."""
    x = Fraction(f) * 2 ** bits / (2 * PI)
    return int(x + Fraction(1, 2))


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 24, 100000])
def test_angles_at_far_positions(pairs, far):
    n, most = len(FREQ), 30000
    place = np.arange(far - most + 1, far + 1)
    pos = []
    for f in FREQ:                                        # nearest to a quarter and to no turn
        per = turns(f, 128)
        frac = np.array([(int(p) * per >> 64) & (2 ** 64 - 1) for p in place], np.uint64).astype(np.float64) * 2.0 ** -64
        pos += [int(place[np.abs(frac - at).argmin()]) for at in (0.25, 0.75, 0.5)] + [int(place[-1])]
    t = len(pos)
    x = torch.zeros(t, 3, 64, dtype=torch.bfloat16, device="cuda")
    x[..., 0:2 * n:2 if pairs else 1][..., :n] = 1.0      # the first value of every pair
    p = ua.Problem(1, 1, 64, 16, 8, 1, 8, t, ua.UA_FLAG_CAUSAL, 0.1)
    p.set_rope(FREQ, ua.UA_ROPE_PAIRS if pairs else ua.UA_ROPE_HALF)
    k = torch.zeros(8, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    slots = torch.arange(t, device="cuda")
    q = p.rope_store(x[:, :1], x[:, 1:2], x[:, 2:], i32(pos), slots, t, k, v)
    assert p.check_device_error() == 0
    for got in (q[:, 0], k.view(-1, 64)[:t]):
        got = got.double().cpu().numpy()
        cos, sin = (got[:, 0:2 * n:2], got[:, 1:2 * n:2]) if pairs else (got[:, :n], got[:, n:2 * n])
        for i, f in enumerate(FREQ):
            per = turns(f, 160)
            for j, at in enumerate(pos):
                # The angle from the nearest quarter turn, exactly, then in double.
                frac = at * per % 2 ** 160
                quarter = (frac + 2 ** 157) >> 158
                rest = 2 * math.pi * math.ldexp(frac - (quarter << 158), -160)
                c, s = math.cos(rest), math.sin(rest)
                want = [(c, s), (-s, c), (-c, -s), (s, -c), (c, s)][quarter]
                off = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + at * 2.0 ** -65)
                for y, w in zip((cos[j, i], sin[j, i]), want):
                    assert abs(y - w) <= off + (2.0 ** -22 + 2.0 ** -8) * abs(w), (f, at, y, w, (y - w) / off)
