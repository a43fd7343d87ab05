"""A cache kept under its budget for good: the totals that a cut returns are the ones that
kv_weights goes on adding to, through the public calls alone.

Tolerances: totals that were copied are equal; what a step adds is held to 1.5e-4 of its
value with the attention call's own lse (1e-4 in the lse, 2e-5 in the sum of exponentials,
as for the single calls), plus half a step of the total it is added to, 2^-24 of it."""
import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.operator_refs import cross_rows, key_weights, keys_to_keep, widen

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hkv,T,lens,budget,row", [
    (2, 40, [40, 7, 0], 8, 8), (2, 40, [40, 7, 0], 8, 9), (4, 600, [600, 512], 512, 700),
    (3, 5000, [5000, 100], 300, 5000),                 # one CTA a row, 1024 threads
    (2, 70000, [70000, 20], 1000, 4096),               # a cluster a row
    (1, 420000, [420000], 2000, 2100),                 # rows longer than the shared memory of a cluster
])
def test_rows_of_totals_with_room(Hkv, T, lens, budget, row):
    r = np.random.default_rng(T + row)
    w = torch.from_numpy(r.standard_exponential((len(lens), Hkv, T), dtype=np.float32)).cuda()
    kept, new, tight = atlas.kv_select(w, ints(lens), budget, keep_first=1, keep_recent=2)
    want = torch.zeros((len(lens), Hkv, row), device="cuda")
    want[..., :budget] = tight
    for b, L in enumerate(lens):
        assert torch.equal(tight[b, 0, :min(L, budget)], w[b, 0][kept[b, 0, :min(L, budget)].long()])
    outs = [atlas.kv_select(w, ints(lens), budget, keep_first=1, keep_recent=2, kept_row_tokens=row)]
    room = torch.full((len(lens) + 1, Hkv, row), 7.0, device="cuda")   # one more: left alone
    outs.append(atlas.kv_select(w, ints(lens), budget, keep_first=1, keep_recent=2, kept_weights=room[:-1]))
    for a, n, x in outs:
        assert torch.equal(a, kept) and torch.equal(n, new) and torch.equal(x, want)
    assert (room[-1] == 7).all()


def test_wrong_rows_and_lengths_in_place_are_refused():
    w, lens = torch.rand((2, 2, 50), device="cuda"), ints([50, 40])
    for kw in (dict(kept_row_tokens=7), dict(kept_weights=torch.empty((2, 2, 7), device="cuda")),
               dict(kept_weights=torch.empty((2, 2, 20), device="cuda"), kept_row_tokens=21),
               dict(kept_weights=torch.empty((2, 1, 20), device="cuda")),
               dict(kept_weights=torch.empty((4, 20), device="cuda"))):
        with pytest.raises(ValueError):
            atlas.kv_select(w, lens, 8, **kw)
    for kw in (dict(new_lens=lens), dict(kept_weights=w)):
        with pytest.raises(atlas.AtlasError):
            atlas.kv_select(w, lens, 8, **kw)
    assert lens.tolist() == [50, 40]


@pytest.mark.parametrize("dtype,Hq,D,P,in_place", [("bf16", 8, 128, 16, True), ("bf16", 2, 64, 64, False),
                                                   ("f32", 2, 64, 16, True), ("f32", 8, 128, 8, False)])
def test_totals_go_on_through_cuts(dtype, Hq, D, P, in_place):
    """Decode steps and cuts in turn; a plain list of (key, total) beside every head."""
    B, Hkv, budget, most, scale = 2, 2, 50, 61, D ** -0.5
    lens = [most, 47]
    r = np.random.default_rng(P)
    width = -(-most // P)
    ids = ints(r.permutation(3 * B * width).tolist())
    tables = [ids[i * B * width:(i + 1) * B * width].reshape(B, width) for i in range(3)]
    kp = torch.zeros((3 * B * width, Hkv, P, D), dtype=DT[dtype], device="cuda")
    vp = kp.clone()

    def rows(H, m):
        return torch.from_numpy(r.standard_normal((B, H, m, D), dtype=np.float32)).to(DT[dtype]).cuda()

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    have, at = ints(lens), 0
    table = tables[at]
    k, v = rows(Hkv, most), rows(Hkv, most)
    atlas.kv_append(k, v, kp, vp, table, ints([0, 0]), have, status=status)
    keys = [[widen(k[b, g, :lens[b]]) for g in range(Hkv)] for b in range(B)]   # what each head holds
    totals = torch.zeros((B, Hkv, width * P), device="cuda")
    for step in range(24):
        if max(have.tolist()) == most:                                          # full: cut to the budget
            before = totals.clone()
            counts = have.tolist()
            kept, have, totals = atlas.kv_select(totals, have, budget, keep_first=2, keep_recent=8,
                                                 kept_row_tokens=width * P, status=status)
            at = at if in_place else (at + 1) % 3
            atlas.kv_compact(kp, vp, table, kept, have, status=status,
                             new_page_table=None if in_place else tables[at])
            table = tables[at]
            for b in range(B):
                n = min(counts[b], budget)
                assert int(have[b]) == n
                for g in range(Hkv):
                    stay = keys_to_keep(before[b, g].tolist(), counts[b], budget, 2, 8)
                    assert kept[b, g, :n].tolist() == stay
                    keys[b][g] = keys[b][g][stay]
                    assert torch.equal(totals[b, g, :n], before[b, g, stay]) and (totals[b, g, n:] == 0).all()
        q, k, v = rows(Hq, 1), rows(Hkv, 1), rows(Hkv, 1)
        atlas.kv_append(k, v, kp, vp, table, have, status=status)
        have = have + 1
        lse = torch.empty((B, Hq, 1), device="cuda")
        atlas.decode(q, kp, vp, table, have, Hq, Hkv, D, P, scale, lse=lse, status=status)
        before = totals.clone()
        assert atlas.kv_weights(q, kp, table, have, lse, Hq, Hkv, D, P, scale, weights=totals,
                                status=status) is totals
        for b in range(B):
            L = int(have[b])
            for g in range(Hkv):
                keys[b][g] = np.concatenate([keys[b][g], widen(k[b, g])])
            kb, qb = np.stack(keys[b])[None], widen(q[b:b + 1])
            add = key_weights(qb, kb, [L], cross_rows(qb, kb, kb, [L], scale)[1], scale)[0]
            grown = widen(totals[b, :, :L]) - widen(before[b, :, :L])
            assert (np.abs(grown - add) <= 1.5e-4 * add + 2.0 ** -24 * widen(totals[b, :, :L])).all()
            assert add.min() > 0 and (totals[b, :, :L] > before[b, :, :L]).float().mean() > 0.5
    assert int(status.item()) == 0
