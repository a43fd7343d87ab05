"""The cache operators as a serving loop uses them, checked step by step against plain
fp64 forms: a prompt rotated into the cache and attended to, its keys' totals, the cut to
a budget (in place and into fresh pages), decode steps that go on from the cut cache at
their true positions, and cross attention to an encoder's pages of the same pool.

Tolerances are those of the single calls: attention 2e-3 (bf16 inputs, fp32 output) and
1e-5 of the largest value (fp32), the weights' 1.5e-4 with the attention call's own lse,
rotated elements 2^-19 (|x| + |y|) and their store."""
import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.gpu_helpers import BF16_ABS, F32_REL
from tests.operator_refs import cross_rows, key_weights, keys_to_keep, row_lse, turned, widen

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gathered(pool, table, b, L):
    """Logical rows [Hkv][L][D] of sequence b, fp64."""
    x = widen(pool[table[b].long()].transpose(0, 1))
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :L]


def near(got, want, dtype):
    tol = F32_REL * np.abs(want).max() if dtype == "f32" else BF16_ABS
    assert np.abs(widen(got) - want).max() <= tol


@pytest.mark.parametrize("dtype,in_place", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_prompt_cut_and_decode(dtype, in_place):
    B, Hq, Hkv, D, P, n, budget, steps = 2, 8, 2, 64, 16, 90, 40, 3
    lens = [90, 71]
    r = np.random.default_rng(11)
    scale = D ** -0.5
    width, enc_pages = 6, 2
    num = B * (width + 3 + enc_pages) + 1
    ids = torch.from_numpy(r.permutation(num).astype(np.int32)).cuda()
    table, fresh, enc_table = (ids[a:z].reshape(B, -1).contiguous() for a, z in (
        (0, B * width), (B * width, B * (width + 3)), (B * (width + 3), num - 1)))
    kp = torch.full((num, Hkv, P, D), float("nan"), dtype=DT[dtype], device="cuda")
    vp = kp.clone()

    def rows(H, m):
        return torch.from_numpy(r.standard_normal((B, H, m, D), dtype=np.float32)).to(DT[dtype]).cuda()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def place(t):  # text with an image inside: time, height, width
        return np.stack([t, t // 8, t % 8])

    axis = atlas.rope_sections((8, 12, 12))
    freq = 1e4 ** (-2.0 * np.arange(32) / 64)

    def angles(t):
        return place(t)[np.array(axis)] * freq

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # ---- the prompts, ragged, into empty caches
    q, k, v = rows(Hq, n), rows(Hkv, n), rows(Hkv, n)
    pos = ints(np.stack([np.stack([place(np.arange(n))[a] for _ in range(B)]) for a in range(3)]).tolist())
    zero, counts = ints([0, 0]), ints(lens)
    qr = atlas.kv_append_rope(q, k, v, kp, vp, table, zero, pos, pair_axis=axis, n_new=counts,
                              q_out=torch.zeros_like(q), status=status)
    for b in range(B):
        got = gathered(kp, table, b, lens[b])
        for t in range(lens[b]):
            x = widen(k[b, :, t])
            tol = 2.0 ** -19 * 2 * np.abs(x).max() + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(got[:, t])
            assert (np.abs(got[:, t] - turned(x, angles(t), False)) <= 1.01 * tol).all()
    # ---- attention over them, and what each key received
    lse = torch.zeros((B, Hq, n), device="cuda")
    out = atlas.prefill(qr, kp, vp, table, counts, Hq, Hkv, D, P, scale, q_lens=counts, lse=lse,
                        out_dtype=torch.float32, status=status)
    w = atlas.kv_weights(qr, kp, table, counts, lse, Hq, Hkv, D, P, scale, q_lens=counts, status=status)
    logical = [(gathered(kp, table, b, lens[b]), gathered(vp, table, b, lens[b])) for b in range(B)]
    for b in range(B):
        kb, vb, qb = logical[b][0][None], logical[b][1][None], widen(qr[b:b + 1, :, :lens[b]])
        exact_lse = row_lse(qb, kb, [lens[b]], scale)
        want = key_weights(qb, kb, [lens[b]], exact_lse, scale)[0]
        assert (np.abs(widen(w[b, :, :lens[b]]) - want) <= 1.5e-4 * want).all()
        for i in (0, lens[b] // 2, lens[b] - 1):
            near(out[b, :, i], cross_rows(qb[:, :, i:i + 1], kb[:, :, :i + 1], vb[:, :, :i + 1], [i + 1], scale)[0][0, :, 0], dtype)
    # ---- the cut
    kept, new, kept_w = atlas.kv_select(w, counts, budget, keep_first=2, keep_recent=8, status=status)
    atlas.kv_compact(kp, vp, table, kept, new, new_page_table=None if in_place else fresh, status=status)
    table = table if in_place else fresh
    assert new.tolist() == [budget, budget]
    cache = []
    for b in range(B):
        ks, vs = [], []
        for g in range(Hkv):
            want = keys_to_keep(w[b, g].tolist(), lens[b], budget, 2, 8)
            assert kept[b, g].tolist() == want
            ks.append(logical[b][0][g][want])
            vs.append(logical[b][1][g][want])
        cache.append((np.stack(ks), np.stack(vs)))
        assert np.array_equal(gathered(kp, table, b, budget), cache[b][0])
        assert np.array_equal(gathered(vp, table, b, budget), cache[b][1])
    # ---- decode goes on: slots from the budget on, positions from the prompt's end on
    have = new.clone()
    totals = torch.zeros((B, Hkv, table.shape[1] * P), device="cuda")
    totals[:, :, :budget] = kept_w
    enc_lens = ints([29, 0])
    ke, ve = rows(Hkv, 29), rows(Hkv, 29)
    atlas.kv_append(ke, ve, kp, vp, enc_table, zero, ints([29, 0]), status=status)
    for step in range(steps):
        q, k, v = rows(Hq, 1), rows(Hkv, 1), rows(Hkv, 1)
        at = [place(np.array(lens[b] + step)) for b in range(B)]
        pos = ints([[[int(at[b][a])] for b in range(B)] for a in range(3)])
        qr = atlas.kv_append_rope(q, k, v, kp, vp, table, have, pos, pair_axis=axis, status=status)
        have = have + 1
        lse = torch.empty((B, Hq, 1), device="cuda")
        out = atlas.decode(qr, kp, vp, table, have, Hq, Hkv, D, P, scale, lse=lse,
                           out_dtype=torch.float32, status=status)
        before = totals.clone()
        atlas.kv_weights(qr, kp, table, have, lse, Hq, Hkv, D, P, scale, weights=totals, status=status)
        crossed = atlas.cross(qr, kp, vp, enc_table, enc_lens, Hq, Hkv, D, P, scale,
                              out_dtype=torch.float32, status=status)
        for b in range(B):
            L = int(have[b])
            kb, vb = gathered(kp, table, b, L), gathered(vp, table, b, L)
            assert np.array_equal(kb[:, :budget], cache[b][0])     # what was kept stays
            qb = widen(qr[b:b + 1])
            ref, ref_lse = cross_rows(qb, kb[None], vb[None], [L], scale)
            near(out[b:b + 1], ref, dtype)
            add = key_weights(qb, kb[None], [L], ref_lse, scale)[0]
            got = widen(totals[b, :, :L]) - widen(before[b, :, :L])
            assert (np.abs(got - add) <= 1.5e-4 * add + 2.0 ** -23 * widen(totals[b, :, :L])).all()
            if b == 0:
                near(crossed[:1], cross_rows(qb, widen(ke[:1]), widen(ve[:1]), [29], scale)[0], dtype)
        assert (crossed[1] == 0).all()
    assert int(status.item()) == 0
