"""README.md's Python examples, run as they stand.  The first against the calls' plain
forms; the second as a loop, its outputs and totals against fp64 on the cache's own keys.

Tolerances: bf16 inputs with a bf16 output 2e-3 plus its store, 2^-8 of the value; a step's
weights 1.5e-4 of their value (the lse's 1e-4 and the sum's 2e-5) and half a step, 2^-24, of
the total they are added to."""
import os
import re

import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.operator_refs import keys_to_keep

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = re.findall(r"^```python\n(.*?)^```", open(os.path.join(ROOT, "README.md")).read(), re.S | re.M)
B, HQ, HKV, D, P = 2, 8, 2, 128, 16


def test_there_are_two_examples_and_they_compile():
    assert len(CODE) == 2
    for text in CODE:
        compile(text, "README.md", "exec")


def rows(H, m, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, H, m, D), generator=g).to(torch.bfloat16).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attended(q, k, v, scale):
    """One head group: q [G][D] over k, v [L][D] in fp64; outputs and weights."""
    p = torch.softmax(q.double() @ k.double().T * scale, -1)
    return p @ v.double(), p


def logical(pool, table, L):
    x = pool[table.long()].transpose(0, 1)
    return x.reshape(HKV, -1, D)[:, :L]


def near(out, want):
    assert ((out.double() - want).abs() <= 2e-3 + 2.0 ** -8 * want.abs()).all()


@pytest.mark.gpu
def test_the_first_example():
    width = 20
    pools = [torch.randn((2 * B * width, HKV, P, D)).to(torch.bfloat16).cuda() for _ in range(2)]
    ids = torch.randperm(2 * B * width).int()
    here, enc = ids[:B * width].reshape(B, width), ids[B * width:].reshape(B, width)
    x = dict(q=rows(HQ, 1, 1), k_pages=pools[0], v_pages=pools[1], page_table=here.cuda(),
             seq_lens=ints([300, 17]), enc_table=enc.cuda(), enc_lens=ints([0, 320]), n_q_heads=HQ,
             n_kv_heads=HKV, head_dim=D, page_tokens=P, scale=D ** -0.5, host_k=pools[0].cpu(),
             host_v=pools[1].cpu(), hot_slots=12, scratch_slots=64, host_page_table=here,
             seq_lens_cpu=torch.tensor([300, 17], dtype=torch.int32))
    exec(CODE[0].replace("out = atlas", "first = atlas"), x)
    for b in range(B):
        for got, table, n in ((x["first"], here, [300, 17]), (x["out"], here, [300, 17]),
                              (x["states"], enc, [0, 320])):
            if n[b] == 0:
                assert (got[b] == 0).all()
                continue
            k, v = (logical(p, table[b].cuda(), n[b]) for p in pools)
            for g in range(HKV):
                heads = slice(g * HQ // HKV, (g + 1) * HQ // HKV)
                near(got[b, heads, 0], attended(x["q"][b, heads, 0], k[g], v[g], D ** -0.5)[0])
    x["pool"].close()


@pytest.mark.gpu
def test_the_second_example_step_after_step():
    n, budget, room = 620, 600, 640
    width = room // P
    kp = torch.zeros((B * width + 1, HKV, P, D), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.randperm(B * width + 1)[:B * width].reshape(B, width).int().cuda()
    k, v = rows(HKV, n, 2), rows(HKV, n, 3)
    time = torch.arange(n, dtype=torch.int32, device="cuda").expand(3, B, n).contiguous()
    counts = ints([n, 580])
    atlas.kv_append_rope(None, k, v, kp, vp, table, ints([0, 0]), time, n_new=counts,
                         pair_axis=atlas.rope_sections((16, 24, 24)))
    x = dict(atlas=atlas, k_pages=kp, v_pages=vp, page_table=table, seq_lens=counts, n_q_heads=HQ,
             n_kv_heads=HKV, head_dim=D, page_tokens=P, scale=D ** -0.5, budget=budget,
             lse=torch.empty((B, HQ, 1), device="cuda"),
             totals=torch.zeros((B, HKV, room), device="cuda"))
    for step in range(25):
        held = x["seq_lens"].tolist()
        x.update(q=rows(HQ, 1, 10 + step), k_new=rows(HKV, 1, 50 + step), v_new=rows(HKV, 1, 90 + step),
                 full=max(held) + 1 == room, positions=ints([[[n + step], [580 + step]]] * 3))
        before = x["totals"].clone()
        if x["full"]:                                  # what the cut will see: a step without it
            y = dict(x, full=False, totals=before.clone(), k_pages=kp.clone(), v_pages=vp.clone())
            exec(CODE[1], y)
        exec(CODE[1], x)
        now = y if x["full"] else x                    # the state before any cut
        for b in range(B):
            L = held[b] + 1
            assert int(now["seq_lens"][b]) == L
            kk, vv = (logical(now[p], table[b], L) for p in ("k_pages", "v_pages"))
            for g in range(HKV):
                heads = slice(g * HQ // HKV, (g + 1) * HQ // HKV)
                want, p = attended(now["q_rot"][b, heads, 0], kk[g], vv[g], D ** -0.5)
                near(now["out"][b, heads, 0], want)
                total, add = now["totals"][b, g, :L].double(), p.sum(0)
                assert ((total - before[b, g, :L].double() - add).abs() <= 1.5e-4 * add + 2.0 ** -24 * total).all()
                if not x["full"]:
                    continue
                stay = keys_to_keep(now["totals"][b, g].tolist(), L, budget, 4, 512)
                assert int(x["seq_lens"][b]) == len(stay) == min(L, budget)
                assert torch.equal(x["totals"][b, g, :len(stay)], now["totals"][b, g, stay])
                assert (x["totals"][b, g, len(stay):] == 0).all()
                for pool, rows_before in ((kp, kk), (vp, vv)):
                    assert torch.equal(logical(pool, table[b], len(stay))[g], rows_before[g][stay])
    assert x["seq_lens"].tolist() == [605, 605]
