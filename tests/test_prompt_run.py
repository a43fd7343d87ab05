"""The operators for batches that share prompts as a serving loop uses them, checked step by step
against plain fp64 forms: pages for the shared prompts and for the sequences from one ring, rows
normed and rotated into them, attention over both, sequences that end and others that take their
places.  And README.md's example of such a step.

Tolerances are those of the single calls: attention 2e-3 (bf16 inputs, fp32 output) and 1e-5 of
the largest value (fp32); normed and rotated elements 2^-18 (|x| + |y|) and their store."""
import os
import re

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.gpu_helpers import BF16_ABS, F32_REL
from tests.operator_refs import turned, widen
from tests.serving_refs import normed, resize, shared_rows

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = re.findall(r"^```py\n(.*?)^```", open(os.path.join(ROOT, "README.md")).read(), re.S | re.M)
EPS, THETA = 1e-6, 1e4


def test_there_is_one_example_and_it_compiles():
    assert len(CODE) == 1
    compile(CODE[0], "README.md", "exec")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gathered(pool, table, L):
    """Logical rows [Hkv][L][D] of one table row, fp64."""
    pages = torch.from_numpy(np.maximum(table, 0)).long().cuda()
    x = widen(pool[pages].transpose(0, 1))
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :L]


def rotated(x, weight, t, D):
    """A token's rows as they should be stored, and the bound |x| + |y| of each element."""
    x = normed(widen(x), widen(weight), EPS, 0.0)
    half = D // 2
    both = np.abs(x[..., :half]) + np.abs(x[..., half:])
    return turned(x, t * THETA ** (-2.0 * np.arange(half) / D), False), np.concatenate([both, both], -1)


def near_rows(got, want, both, dtype):
    store = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert (np.abs(got - want) <= 2.0 ** -18 * both + store * np.abs(want)).all()


class Tables:
    """One kv_resize batch on both sides; the ring and its state are shared by several."""

    def __init__(self, B, width, ring):
        self.table, self.held, self.ring = np.full((B, width), -1, np.int32), [0] * B, ring
        self.dev = ints(self.table.tolist()), ints(self.held)

    def resize(self, lens, P, n_new=None, max_new=0):
        status = ints([0])
        slots = atlas.kv_resize(*self.dev, ints(lens), self.ring["ids"], self.ring["state"], P,
                                n_new=None if n_new is None else ints(n_new),
                                max_new=max_new or None, status=status)
        want = resize(self.table, self.held, lens, self.ring["plain"][0], self.ring["plain"][1], P, n_new, max_new)
        self.table, self.held = want[:2]
        self.ring["plain"] = want[2], want[3]
        for got, x in zip((*self.dev, self.ring["ids"], self.ring["state"]), want):
            assert np.array_equal(got.cpu().numpy(), np.array(x))
        assert int(status.item()) == want[5] == 0
        if max_new:
            assert np.array_equal(slots.cpu().numpy(), want[4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,path", [("bf16", 128, 0), ("bf16", 64, 8), ("bf16", 128, 24), ("f32", 64, 0)])
def test_prompts_steps_ends_and_arrivals(dtype, D, path):
    Hq, Hkv, P, N, width = 8, 2, 16, 60, 6
    B, starts, prefix = 6, [0, 3, 5], [70, 33]                 # (the last sequence shares none)
    r = np.random.default_rng(31)
    scale = D ** -0.5
    status = ints([0])
    ids = r.permutation(N).tolist()
    ring = dict(ids=ints(ids), state=ints([17, N]), plain=(ids, [17, N]))
    kp = torch.full((N, Hkv, P, D), float("nan"), dtype=DT[dtype], device="cuda")
    vp = kp.clone()
    wq, wk = (torch.from_numpy(r.uniform(0.5, 1.5, D).astype(np.float32)).to(DT[dtype]).cuda() for _ in range(2))
    kw = dict(q_weight=wq, k_weight=wk, eps=EPS, theta=THETA, status=status)

    def rows(batch, H, m):
        return torch.from_numpy(r.standard_normal((batch, H, m, D), dtype=np.float32)).to(DT[dtype]).cuda()

    # ---- the shared prompts
    shared, own = Tables(2, 5, ring), Tables(B, width, ring)
    shared.resize(prefix, P)
    k, v = rows(2, Hkv, 70), rows(2, Hkv, 70)
    time = torch.arange(70, dtype=torch.int32, device="cuda").expand(1, 2, 70).contiguous()
    assert atlas.kv_append_norm_rope(None, k, v, kp, vp, shared.dev[0], ints([0, 0]), time,
                                     n_new=ints(prefix), **kw) is None
    parts = []
    for g in range(2):
        got = gathered(kp, shared.table[g], prefix[g]), gathered(vp, shared.table[g], prefix[g])
        for t in range(prefix[g]):
            near_rows(got[0][:, t], *rotated(k[g, :, t], wk, t, D), dtype)
        assert np.array_equal(got[1], widen(v[g, :, :prefix[g]]))
        parts.append(got)
    before = [prefix[0]] * 3 + [prefix[1]] * 2 + [0]           # a sequence's first position

    # ---- the sequences: prompts of their own, then steps, some of which end or begin one
    lens = [0] * B
    steps = [[12, 4, 1, 9, 0, 3]] + [[1] * B for _ in range(9)]
    steps[3] = [1, 0, 1, 1, 0, 1]                              # two places are idle
    steps[4] = [4, 7, 1, 2, 5, 1]                              # new prompts, drafts
    for now, counts in enumerate(steps):
        if now == 3:
            lens[1] = 0                                        # its pages go back to the ring
        if now == 7:
            lens[3], counts = 0, [1, 1, 1, 20, 1, 0]           # taken over in the same step
        n = max(counts)
        past = list(lens)
        lens = [a + c for a, c in zip(past, counts)]
        if now == 3:
            own.resize(lens, P)
        else:
            own.resize(lens, P, counts, n)
        q, k, v = rows(B, Hq, n), rows(B, Hkv, n), rows(B, Hkv, n)
        pos = ints([[[before[b] + past[b] + i for i in range(n)] for b in range(B)]])
        q_rot = atlas.kv_append_norm_rope(q, k, v, kp, vp, own.dev[0], ints(past), pos,
                                          n_new=ints(counts), q_out=torch.zeros_like(q), **kw)
        lse = torch.zeros((B, Hq, n), device="cuda")
        out = atlas.shared(q_rot, kp, vp, shared.dev[0], ints(prefix), ints(starts), own.dev[0], ints(lens),
                           Hq, Hkv, D, P, scale, q_lens=ints(counts), lse=lse, out_dtype=torch.float32,
                           status=status, debug_flags=path)
        assert int(status.item()) == 0
        kl, vl = np.zeros((B, Hkv, width * P, D)), np.zeros((B, Hkv, width * P, D))
        for b in range(B):
            kl[b, :, :lens[b]] = gathered(kp, own.table[b], lens[b])
            vl[b, :, :lens[b]] = gathered(vp, own.table[b], lens[b])
            for i in range(counts[b]):
                t = before[b] + past[b] + i
                near_rows(kl[b, :, past[b] + i], *rotated(k[b, :, i], wk, t, D), dtype)
                near_rows(widen(q_rot[b, :, i]), *rotated(q[b, :, i], wq, t, D), dtype)
                assert np.array_equal(vl[b, :, past[b] + i], widen(v[b, :, i]))
        ref, ref_lse = shared_rows(widen(q_rot), parts, starts, kl, vl, lens, scale, counts)
        real = ~np.isnan(ref_lse)
        tol = F32_REL * np.abs(ref[real]).max() if dtype == "f32" else BF16_ABS
        assert np.abs(widen(out)[real] - ref[real]).max() <= tol
        assert np.abs(widen(lse)[real] - ref_lse[real]).max() <= (2e-5 if dtype == "f32" else 1e-4)
    for t in (own, shared):
        t.resize([0] * len(t.held), P)
    assert ring["plain"][1][1] == N and sorted(ring["ids"].tolist()) == list(range(N))


@pytest.mark.gpu
def test_the_example():
    Hq, Hkv, D, P, B, N = 8, 2, 128, 16, 3, 40
    g = torch.Generator().manual_seed(4)

    def rows(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()

    kp, vp = rows(N, Hkv, P, D), rows(N, Hkv, P, D)
    w = torch.linspace(0.5, 1.5, D).to(torch.bfloat16).cuda()
    ring, plain = list(range(4, N)) + [-1] * 4, [0, N - 4]     # pages 0 to 3 hold the prompt
    x = dict(atlas=atlas, k_pages=kp, v_pages=vp, prefix_table=ints([[0, 1, 2, 3]]), prefix_lens=ints([60]),
             group_starts=ints([0, B]), page_table=ints([[-1] * 4] * B), n_pages=ints([0] * B),
             free_pages=ints(ring), free_state=ints(plain), seq_lens=ints([0] * B), n_q_heads=Hq,
             n_kv_heads=Hkv, head_dim=D, page_tokens=P, scale=D ** -0.5, q_weight=w, k_weight=w.flip(0))
    prompt = [(gathered(kp, np.arange(4), 60), gathered(vp, np.arange(4), 60))]
    table, held = np.full((B, 4), -1, np.int32), [0] * B
    for step in range(20):
        x.update(q=rows(B, Hq, 1, D), k_new=rows(B, Hkv, 1, D), v_new=rows(B, Hkv, 1, D))
        exec(CODE[0], x)
        lens = [step + 1] * B
        table, held, ring, plain, _, _ = resize(table, held, lens, ring, plain, P)
        assert np.array_equal(x["page_table"].cpu().numpy(), table) and x["seq_lens"].tolist() == lens
        k, v = (np.stack([gathered(p, table[b], step + 1) for b in range(B)]) for p in (kp, vp))
        for b in range(B):
            near_rows(k[b, :, step], *rotated(x["k_new"][b, :, 0], w.flip(0), 60 + step, D), "bf16")
            near_rows(widen(x["q_rot"][b, :, 0]), *rotated(x["q"][b, :, 0], w, 60 + step, D), "bf16")
        ref, _ = shared_rows(widen(x["q_rot"]), prompt, [0, B], k, v, lens, D ** -0.5)
        assert (np.abs(widen(x["out"]) - ref) <= 2e-3 + 2.0 ** -8 * np.abs(ref)).all()
