"""Plain fp64 forms of the cache operators, for the tests: numpy on logical (unpaged)
arrays, one row at a time, with nothing of the library's.  Paging is tests/paging.py's."""
import math
from fractions import Fraction

import numpy as np


def widen(t):
    """The exact values of a torch tensor (any float type) as fp64 numpy."""
    return t.detach().cpu().double().numpy()


TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")


def angle(position, freq):
    """position * freq (an int and a double) modulo a turn, exact to the last bit of a double."""
    return float(Fraction(int(position)) * Fraction(freq) % TWO_PI)


def cross_rows(q, k, v, lens, scale, q_lens=None, sinks=None, softcap=0.0):
    """q [B][Hq][n][D]; k, v [B][Hkv][T][D]; lens [B].  out, lse; rows >= q_lens[b] NaN."""
    B, Hq, n, D = q.shape
    G = Hq // k.shape[1]
    out = np.full(q.shape, np.nan)
    lse = np.full((B, Hq, n), np.nan)
    for b in range(B):
        for h in range(Hq):
            for i in range(n if q_lens is None else q_lens[b]):
                s = scale * (k[b, h // G, : lens[b]] @ q[b, h, i])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                extra = [] if sinks is None else [float(sinks[h])]
                m = max(list(s) + extra, default=-math.inf)
                if m == -math.inf:
                    out[b, h, i], lse[b, h, i] = 0.0, -math.inf
                    continue
                p = np.exp(s - m)
                total = p.sum() + sum(math.exp(x - m) for x in extra)
                out[b, h, i] = p @ v[b, h // G, : lens[b]] / total
                lse[b, h, i] = m + math.log(total)
    return out, lse


def pair_elements(pairs, interleaved):
    a = np.arange(pairs) * 2 if interleaved else np.arange(pairs)
    return a, a + 1 if interleaved else a + pairs


def turned(x, angles, interleaved):
    """Rows x [..., D] with their first 2 * len(angles) elements turned by angles."""
    a, b = pair_elements(len(angles), interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * np.cos(angles) - x[..., b] * np.sin(angles)
    y[..., b] = x[..., b] * np.cos(angles) + x[..., a] * np.sin(angles)
    return y
