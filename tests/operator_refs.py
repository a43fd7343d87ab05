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


def key_weights(q, k, lens, lse, scale, q_lens=None, window=0, softcap=0.0):
    """What atlas_kv_weights adds: [B][Hkv][T] in fp64, 0 for keys nobody sees."""
    B, Hq, n, D = q.shape
    Hkv, T = k.shape[1:3]
    w = np.zeros((B, Hkv, T))
    for b in range(B):
        rows = n if q_lens is None else q_lens[b]
        for h in range(Hq):
            for i in range(rows):
                if lse[b, h, i] == -math.inf:
                    continue
                end = lens[b] - rows + i + 1
                start = max(0, end - window) if window else 0
                g = h // (Hq // Hkv)
                s = scale * (k[b, g, start:end] @ q[b, h, i])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                w[b, g, start:end] += np.exp(s - lse[b, h, i])
    return w


def row_lse(q, k, lens, scale, q_lens=None, window=0, softcap=0.0):
    """The log-sum-exp of each causal row, fp64; rows >= q_lens[b] NaN."""
    B, Hq, n, D = q.shape
    lse = np.full((B, Hq, n), np.nan)
    for b in range(B):
        rows = n if q_lens is None else q_lens[b]
        for h in range(Hq):
            for i in range(rows):
                end = lens[b] - rows + i + 1
                start = max(0, end - window) if window else 0
                s = scale * (k[b, h * k.shape[1] // Hq, start:end] @ q[b, h, i])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                lse[b, h, i] = s.max() + math.log(np.exp(s - s.max()).sum())
    return lse


def keys_to_keep(w, L, budget, first, recent):
    """Indices that stay of one row of totals, by the rule of atlas_kv_select."""
    if L <= budget:
        return list(range(L))
    must = [t for t in range(L) if t < first or t >= L - recent]
    rest = [t for t in range(first, L - recent)]
    value = [-math.inf if math.isnan(w[t]) else w[t] for t in range(L)]
    rest.sort(key=lambda t: (-value[t], t))
    return sorted(must + rest[: budget - len(must)])
