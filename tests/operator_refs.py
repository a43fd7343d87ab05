"""Plain fp64 forms of the cache operators, for the tests: numpy on logical (unpaged)
arrays, one row at a time, with nothing of the library's.  Paging is tests/paging.py's."""
import math

import numpy as np


def widen(t):
    """The exact values of a torch tensor (any float type) as fp64 numpy."""
    return t.detach().cpu().double().numpy()


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
