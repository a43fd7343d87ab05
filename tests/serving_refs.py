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


def normed(x, weight, eps, offset):
    """Rows x [..., D] over their root mean square, times weight + offset."""
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (weight + offset)


def resize(table, held, lens, ring, state, P, n_new=None, max_new=0):
    """atlas_kv_resize, one sequence after the other, on copies: the table, n_pages, ring, state
    and slots after it, and the status bits."""
    table, held, ring = table.copy(), list(held), list(ring)
    B, width = table.shape
    N, (head, count) = len(ring), state
    slots, bits = np.full((B, max_new), -1, np.int32), 0

    def fresh(b):
        return 0 if not max_new else n_new[b] if n_new is not None else min(max_new, max(lens[b], 0))

    def bad(b):
        return not (0 <= lens[b] <= width * P and 0 <= held[b] <= width and
                    0 <= fresh(b) <= min(max_new, lens[b]))

    want = [held[b] if bad(b) else -(-lens[b] // P) for b in range(B)]
    if any(bad(b) for b in range(B)):
        bits |= 2
    back = sum(max(0, held[b] - want[b]) for b in range(B))
    if not (0 <= head < N and 0 <= count <= N) or count + back > N:
        return table, held, ring, list(state), slots, bits | 1
    asked = taken = given = 0
    moved = list(held)
    for b in range(B):
        asked += max(0, want[b] - held[b])
        if want[b] > held[b] and asked > count:
            bits |= 8
            continue
        for j in range(held[b], want[b]):
            table[b, j] = ring[(head + taken) % N]
            taken += 1
        for j in range(want[b], held[b]):
            ring[(head + count + given) % N] = table[b, j]
            table[b, j] = -1
            given += 1
        moved[b] = want[b]
        if bad(b):
            continue
        for i in range(fresh(b)):
            t = lens[b] - fresh(b) + i
            slots[b, i] = table[b, t // P] * P + t % P
    return table, moved, ring, [(head + taken) % N, count - taken + given], slots, bits
