"""Plain fp64 forms of the operators for batches that share prompts, for the tests: numpy on
logical (unpaged) arrays, one row or one sequence at a time, with nothing of the library's."""
import math

import numpy as np


def shared_rows(q, prefixes, starts, k, v, lens, scale, q_lens=None, sinks=None, softcap=0.0):
    """q [B][Hq][n][D]; prefixes: a (k, v) of [Hkv][T][D] for each group; k, v: the sequences'
    own, [B][Hkv][T][D], of which lens[b] count.  out, lse; rows >= q_lens[b] NaN."""
    B, Hq, n, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full(q.shape, np.nan), np.full((B, Hq, n), np.nan)
    for b in range(B):
        rows = n if q_lens is None else q_lens[b]
        mine = [g for g in range(len(prefixes)) if starts[g] <= b < starts[g + 1]]
        for h in range(Hq):
            parts = [(pk[h // G], pv[h // G]) for pk, pv in (prefixes[g] for g in mine)]
            for i in range(rows):
                end = lens[b] - rows + i + 1
                keys = np.concatenate([p[0] for p in parts] + [k[b, h // G, :end]])
                vals = np.concatenate([p[1] for p in parts] + [v[b, h // G, :end]])
                s = scale * (keys @ q[b, h, i])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                extra = [] if sinks is None else [float(sinks[h])]
                m = max(list(s) + extra)
                p = np.exp(s - m)
                total = p.sum() + sum(math.exp(x - m) for x in extra)
                out[b, h, i] = p @ vals / total
                lse[b, h, i] = m + math.log(total)
    return out, lse
