"""The angles of the rotary append themselves: rows (1, 0) and (0, 1) of every pair come out
as (cos, sin) and (-sin, cos).

Tolerance against the exact angle: 2^-24 turns (2 pi of them in radians), the fp32 form of at
most an eighth of a turn (pi / 4 2^-24), 2^-32 turns dropped, and sincospif's 2 ulp of a value
below 1 (2 * 2^-24).  The products with 1 and 0 and their sum are exact.

Frequencies of both signs: f and -f turn by the same angle either way but for one step of
2^-32 turns, so their fp32 forms are at most one step apart (pi 2^-26) and each value within
2 ulp: 2^-22 + pi 2^-26, next to 1.5 * 2^-24 turns (5.6e-7) for a frequency that is reduced
to the whole turn below it."""
import math

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.operator_refs import angle, widen

pytestmark = pytest.mark.gpu
FAR = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1 << 30, -(10 ** 9), 123456789, 10 ** 6, -4097, 1, 0]
EXACT = 2 * math.pi * (2.0 ** -24 + 2.0 ** -32) + math.pi / 4 * 2.0 ** -24 + 2 * 2.0 ** -24
MIRROR = 2.0 ** -22 + math.pi * 2.0 ** -26 + 2 * math.pi * 2.0 ** -32


def cos_sin(freq, interleaved, D=128, P=16):
    """[positions][pairs] cosines and sines of the kernel, from the rotated queries."""
    pairs, n = len(freq), len(FAR)
    q = torch.zeros((1, 2, n, D), device="cuda")
    first = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    second = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    q[0, 0, :, first] = 1
    q[0, 1, :, second] = 1
    kv = torch.zeros((1, 1, n, D), device="cuda")
    pool = torch.zeros((2, 1, P, D), device="cuda")
    out = atlas.kv_append_rope(q, kv, kv, pool, pool.clone(), torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.tensor([FAR], dtype=torch.int32, device="cuda"), inv_freq=freq,
                               rot_dim=2 * pairs, interleaved=interleaved)
    x = widen(out)[0]
    assert np.array_equal(x[0, :, first], x[1, :, second]) and np.array_equal(x[0, :, second], -x[1, :, first])
    return x[0, :, first], x[0, :, second]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("theta,pairs", [(1e6, 64), (1e4, 32), (1e4, 63), (5e5, 48)])
def test_angles_of_either_sign_at_any_position(theta, pairs, sign, interleaved):
    freq = [sign * theta ** (-p / pairs) for p in range(pairs)]
    cos, sin = cos_sin(freq, interleaved)
    z = np.array([[angle(t, f) for f in freq] for t in FAR])
    assert np.abs(cos - np.cos(z)).max() <= EXACT and np.abs(sin - np.sin(z)).max() <= EXACT
    assert (cos[-1] == 1).all() and (sin[-1] == 0).all()              # position 0


@pytest.mark.parametrize("theta,pairs", [(1e6, 64), (1e4, 63)])
def test_a_negative_frequency_mirrors_the_positive_one(theta, pairs):
    freq = [theta ** (-p / pairs) for p in range(pairs)]
    cos, sin = cos_sin(freq, False)
    cos_n, sin_n = cos_sin([-f for f in freq], False)
    assert np.abs(cos - cos_n).max() <= MIRROR and np.abs(sin + sin_n).max() <= MIRROR
