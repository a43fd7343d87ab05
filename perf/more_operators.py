"""Serving a batch of requests that share prompts, as measured work: what a case is, its
inputs, one pass through it, and what that pass has to read, write and compute.

Three operators over the page pools [num_pages][Hkv][P][D] of the library:

  shared     attention of a batch whose sequences share long prefixes in groups: a prefix's
             pages are there once, and each sequence has a cache of its own behind it;
  norm_rope  a root-mean-square norm of each head's queries and keys, then their rotary
             positions, while the keys and values go into their pages;
  resize     page tables and slots made from the requests' lengths: each sequence takes the
             pages that it lacks from a ring of free ones or gives back what it has too many.

``own`` selects the library's calls; otherwise ``run`` computes the operators in plain
torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decode step of a few requests behind a system prompt (latency)
        dict(name="shared_step_few", op="shared", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, P=16,
             q=1, groups=1, prefix=1024, own_lo=1, own_hi=128, lens_seed=1, bare=False,
             ragged=False, sinks=False, softcap=0.0),
        # a serving batch that asks about one long document
        dict(name="shared_step_document", op="shared", dtype="bf16", B=64, Hq=32, Hkv=8, D=128,
             P=16, q=1, groups=1, prefix=32768, own_lo=1, own_hi=2048, lens_seed=2, bare=False,
             ragged=False, sinks=False, softcap=0.0),
        # many requests over several prompts of all lengths, one group without any; each
        # checks a few drafted tokens
        dict(name="shared_draft_groups", op="shared", dtype="bf16", B=192, Hq=32, Hkv=8, D=128,
             P=64, q=4, groups=7, prefix=16001, own_lo=4, own_hi=1000, lens_seed=3, bare=True,
             ragged=True, sinks=False, softcap=0.0),
        # fp32, small heads
        dict(name="shared_step_f32", op="shared", dtype="f32", B=16, Hq=16, Hkv=4, D=64, P=32,
             q=1, groups=2, prefix=4000, own_lo=1, own_hi=500, lens_seed=4, bare=False,
             ragged=False, sinks=True, softcap=0.0),
        # the requests' own prompts behind a shared one
        dict(name="shared_prompts", op="shared", dtype="bf16", B=16, Hq=32, Hkv=8, D=128, P=16,
             q=256, groups=1, prefix=8192, own_lo=256, own_hi=300, lens_seed=5, bare=False,
             ragged=True, sinks=False, softcap=0.0),
        # a decode step: one token per sequence, normed, rotated and written
        dict(name="norm_rope_step", op="norm_rope", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=16,
             n=1, past=4000, rot=128, interleaved=False, fused=True, ragged=False, per_head=False,
             offset=0.0, theta=1000000.0, far=3000),
        # fp32 prompts, half a head rotated, pairs side by side, weights stored less one
        dict(name="norm_rope_part_f32", op="norm_rope", dtype="f32", B=3, Hq=16, Hkv=4, D=64, P=32,
             n=777, past=13, rot=32, interleaved=True, fused=False, ragged=True, per_head=True,
             offset=1.0, theta=10000.0, far=0),
        # long prompts straight from the fused projection
        dict(name="norm_rope_prompts", op="norm_rope", dtype="bf16", B=4, Hq=32, Hkv=8, D=128,
             P=64, n=8192, past=0, rot=128, interleaved=False, fused=True, ragged=False,
             per_head=False, offset=0.0, theta=1000000.0, far=0),
        # a batch makes room for drafted tokens and gives back what was not accepted (latency)
        dict(name="resize_draft", op="resize", B=32, P=16, lo=1000, hi=32768, lens_seed=6,
             draft=8, turnover=0.0, slots=8),
        # requests come and go, the room for their prompts with them
        dict(name="resize_arrivals", op="resize", B=64, P=16, lo=1, hi=32768, lens_seed=7,
             draft=1, turnover=0.5, slots=2048),
        # a large pool under a long-context load
        dict(name="resize_long", op="resize", B=256, P=16, lo=1, hi=131072, lens_seed=8, draft=1,
             turnover=0.5, slots=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the listed ranges.  One that would need more than its operator's
    largest listed case gets a smaller batch, then shorter sequences."""
    op = rng.choice(["shared", "shared", "norm_rope", "resize"])
    if op == "resize":
        hi = _log_int(rng, 16, 131072)
        c = dict(op=op, B=_log_int(rng, 1, 1024), P=rng.choice([8, 16, 32, 64, 128]),
                 lo=rng.choice([0, 1, hi // 2 + 1]), hi=hi, lens_seed=rng.randrange(1 << 20),
                 draft=_log_int(rng, 1, 64), turnover=rng.choice([0.0, 0.1, 0.5]),
                 slots=rng.choice([0, 1, _log_int(rng, 2, 4096)]))
    else:
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), D=D, Hkv=Hkv,
                 Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), P=rng.choice([8, 16, 32, 64, 128]))
        if op == "shared":
            B = _log_int(rng, 1, 256)
            q = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 300)])
            hi = _log_int(rng, max(2, q), max(2 * q, 4096))
            c.update(B=B, q=q, groups=min(B, _log_int(rng, 1, 16)), prefix=_log_int(rng, 16, 32768),
                     own_lo=q, own_hi=hi, lens_seed=rng.randrange(1 << 20),
                     bare=rng.random() < 0.3, ragged=rng.random() < 0.4,
                     sinks=rng.random() < 0.3, softcap=rng.choice([0.0, 0.0, 0.0, 30.0]))
        else:
            c.update(B=_log_int(rng, 1, 32), n=rng.choice([1, _log_int(rng, 2, 8192)]),
                     past=rng.randrange(0, 3000), rot=rng.choice([D, D, D // 2, 24, 6]),
                     interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                     ragged=rng.random() < 0.4, per_head=rng.random() < 0.3,
                     offset=rng.choice([0.0, 0.0, 1.0]), theta=rng.choice([10000.0, 1000000.0]),
                     far=rng.choice([0, 0, _log_int(rng, 1000, 1000000)]))
    most = {k: max(work(x)[k] for x in listed() if x["op"] == op) for k in ("bytes", "flops")}
    while any(work(c)[k] > most[k] for k in most):
        if c["B"] > 1:
            c["B"] = c["B"] // 2
            if op == "shared":
                c["groups"] = min(c["groups"], c["B"])
        elif op == "norm_rope":
            c["n"] //= 2
        elif op == "shared":
            c["prefix"] = c["prefix"] // 2
        else:
            c["slots"] //= 2
            c["hi"] //= 2
            c["lo"] = min(c["lo"], c["hi"])
    return c


def _rows(c, n):
    """Rows of each sequence: n, or up to n (the last sequence short) in a ragged batch."""
    return np.array([n] + [max(1, n - (b * 37) % n) for b in range(1, c["B"])]) \
        if c["ragged"] else np.full(c["B"], n)


def _shared_lens(c):
    """Own lengths [B], group borders [groups + 1] and prefix lengths [groups] of a case."""
    r = random.Random(c["lens_seed"])
    B, n = c["B"], c["groups"]
    lens = np.array([r.randint(c["own_lo"], c["own_hi"]) for _ in range(B)])
    lens[0] = c["own_hi"]
    starts = np.array([0] + sorted(r.sample(range(1, B), n - 1)) + [B])
    prefix = np.array([r.randint(c["prefix"] // 8 + 1, c["prefix"]) for _ in range(n)])
    prefix[0] = c["prefix"]
    if c["bare"] and n > 1:
        prefix[-1] = 0
    return lens, starts, prefix


def _resize_lens(c):
    """The lengths of the sequences now, in the first step and in the second, [B] each."""
    r = random.Random(c["lens_seed"])
    now, first, second = [], [], []
    for b in range(c["B"]):
        x = r.randint(c["lo"], c["hi"])
        if r.random() < c["turnover"]:  # a request ends in one step, another comes in the other
            a, z = (0, x) if r.random() < 0.5 else (r.randint(c["lo"], c["hi"]), 0)
        else:                           # a request goes on: some of the drafted tokens stay
            a, z = x + c["draft"], x + r.randint(0, c["draft"])
        now.append(z)
        first.append(a)
        second.append(z)
    return np.array(now), np.array(first), np.array(second)


def work(case):
    c = case
    if c["op"] == "resize":
        now, first, _ = _resize_lens(c)
        moved = int(np.abs(-(-first // c["P"]) + (-now // c["P"])).sum())
        # a page taken: read from the ring, written to the table; given back: read from the
        # table, written to the ring, its place in the table cleared.  Each moves once each way.
        new = 2 * c["slots"] * c["B"]
        return {"bytes": 4 * (5 * moved + new + 2 * 4 * c["B"]), "flops": 2 * (moved + new + c["B"])}
    e = _BYTES[c["dtype"]]
    D = c["D"]
    if c["op"] == "norm_rope":
        rows = int(_rows(c, c["n"]).sum())
        moved = 2 * rows * (c["Hq"] + 2 * c["Hkv"]) * D * e
        return {"bytes": moved + 4 * rows, "flops": rows * (c["Hq"] + c["Hkv"]) * (4 * D + 3 * c["rot"])}
    lens, starts, prefix = _shared_lens(c)
    rows = _rows(c, c["q"])
    per_seq = np.repeat(prefix, np.diff(starts))
    pairs = c["Hq"] * int((rows * (per_seq + lens) - rows * (rows - 1) // 2).sum())
    return {"bytes": 2 * int(lens.sum() + prefix.sum()) * c["Hkv"] * D * e
            + 2 * int(rows.sum()) * c["Hq"] * D * e + 4 * int(rows.sum()) * c["Hq"],
            "flops": pairs * (4 * D + 4)}


def _tensor(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _table(perm, pages, base):
    """Rows of page ids from perm[base:], pages[b] each; what lies behind them is 0."""
    width = max(1, int(pages.max()))
    first = np.concatenate([[0], np.cumsum(pages)])[:-1] + base
    at = torch.from_numpy(first[:, None] + np.arange(width)[None]).cuda()
    inside = torch.from_numpy(np.arange(width)[None] < pages[:, None]).cuda()
    return torch.where(inside, perm[at.clamp(max=perm.numel() - 1)], 0).to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] == "resize":
        B, P = c["B"], c["P"]
        now, first, second = _resize_lens(c)
        held, most = -(-now // P), -(-first // P)
        num = int(held.sum() + np.maximum(most - held, 0).sum()) + 5
        perm = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        width = int(max(held.max(), most.max(), 1)) + 1
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        rows = _table(perm, held, 0)
        inside = torch.from_numpy(np.arange(rows.shape[1])[None] < held[:, None]).cuda()
        table[:, : rows.shape[1]] = torch.where(inside, rows, -1)
        s["table"], s["n_pages"] = table, _tensor(held)
        head = int(torch.randint(0, num, (1,), generator=g, device="cuda"))
        free = perm[int(held.sum()):]
        ring = torch.full((num,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(free.numel(), device="cuda")) % num] = free
        s["ring"], s["free"] = ring, _tensor([head, free.numel()])
        s["steps"] = []
        for to, before in ((first, second), (second, first)):
            new = np.minimum(np.maximum(to - before, 0), c["slots"])
            s["steps"].append((_tensor(to), _tensor(new) if c["slots"] else None,
                               torch.zeros((B, c["slots"]), dtype=torch.int32, device="cuda")
                               if c["slots"] else None))
        return s
    dt = _DT[c["dtype"]]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if c["op"] == "shared":
        lens, starts, prefix = _shared_lens(c)
        own_pages, shared_pages = -(-lens // P), -(-prefix // P)
        num = int(own_pages.sum() + shared_pages.sum()) + 3
        # every page has one owner; what lies behind a sequence's end is stale data
        perm = torch.randperm(num, generator=g, device="cuda")
        s["table"] = _table(perm, own_pages, 0)
        s["prefix_table"] = _table(perm, shared_pages, int(own_pages.sum()))
        s["lens"], s["starts"], s["prefix_lens"] = _tensor(lens), _tensor(starts), _tensor(prefix)
        s["k_pages"], s["v_pages"] = normal(num, Hkv, P, D), normal(num, Hkv, P, D)
        s["q_rows"] = normal(B, Hq, c["q"], D)
        s["q_lens"] = _tensor(_rows(c, c["q"])) if c["ragged"] else None
        s["scale"] = 1.0 / math.sqrt(D)
        s["sink"] = torch.randn(Hq, generator=g, device="cuda") if c["sinks"] else None
        s["out"] = torch.zeros((B, Hq, c["q"], D), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((B, Hq, c["q"]), device="cuda")
        return s
    n = c["n"]
    past = np.full(B, c["past"]) + np.arange(B) % 7
    pages = -(-(past + n) // P)
    num = int(pages.sum()) + 3
    s["table"] = _table(torch.randperm(num, generator=g, device="cuda"), pages, 0)
    s["k_pages"], s["v_pages"] = normal(num, Hkv, P, D), normal(num, Hkv, P, D)
    # what a projection gives: heads of different sizes
    size = torch.exp(torch.randn((1, Hq + 2 * Hkv, 1, 1), generator=g, device="cuda")).to(dt)
    if c["fused"]:  # one projection's output, token after token
        qkv = (normal(B, n, Hq + 2 * Hkv, D) * size.transpose(1, 2)).transpose(1, 2)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"], s["k_new"], s["v_new"] = (normal(B, h1 - h0, n, D) * size[:, h0:h1] for h0, h1 in (
            (0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    s["q_out"] = torch.zeros((B, Hq, n, D), dtype=dt, device="cuda")
    s["past_lens"] = _tensor(past)
    s["n_new"] = _tensor(_rows(c, n)) if c["ragged"] else None
    s["positions"] = (torch.arange(n, device="cuda") + s["past_lens"][:, None] + c["far"]).to(torch.int32)
    for name, H in (("q_weight", Hq), ("k_weight", Hkv)):
        shape = (H, D) if c["per_head"] else (D,)
        w = 1.0 - c["offset"] + 0.2 * torch.randn(shape, generator=g, device="cuda")
        s[name] = w.to(dt)
    s["eps"] = 1e-6
    return s


def run(state):
    s = state
    if own:
        return _own(s)
    return {"shared": _shared, "norm_rope": _norm_rope, "resize": _resize}[s["op"]](s)


def _own(s):
    import exact_causal_gqa_gb300 as atlas
    if s["op"] == "shared":
        out = atlas.shared(s["q_rows"], s["k_pages"], s["v_pages"], s["prefix_table"],
                           s["prefix_lens"], s["starts"], s["table"], s["lens"], s["Hq"], s["Hkv"],
                           s["D"], s["P"], s["scale"], out=s["out"], lse=s["lse"],
                           q_lens=s["q_lens"], sinks=s["sink"], softcap=s["softcap"])
        return {"out": out, "lse": s["lse"]}
    if s["op"] == "norm_rope":
        q = atlas.kv_append_norm_rope(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"],
                                      s["table"], s["past_lens"], s["positions"],
                                      q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                      weight_offset=s["offset"], theta=s["theta"], rot_dim=s["rot"],
                                      interleaved=s["interleaved"], n_new=s["n_new"], q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    for lens, new, slots in s["steps"]:
        atlas.kv_resize(s["table"], s["n_pages"], lens, s["ring"], s["free"], s["P"], n_new=new,
                        slots=slots)
    return _resized(s)


def _resized(s):
    out = {"table": s["table"], "n_pages": s["n_pages"], "ring": s["ring"], "free": s["free"]}
    if s["slots"]:
        out.update(first=s["steps"][0][2], second=s["steps"][1][2])
    return out


def _logical(pages, table):
    """[num_pages][Hkv][P][D] through the table -> [B][Hkv][width * P][D] in fp32."""
    x = pages[table.long()].transpose(1, 2).float()
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _shared(s):
    B, Hq, q, D = s["q_rows"].shape
    Hkv = s["Hkv"]
    G = Hq // Hkv
    qf = s["q_rows"].float().reshape(B, Hkv, G * q, D) * s["scale"]

    def scores(rows, k):
        x = torch.matmul(rows, k.transpose(-1, -2))
        return s["softcap"] * torch.tanh(x / s["softcap"]) if s["softcap"] else x

    # each sequence over its own keys
    k, v = _logical(s["k_pages"], s["table"]), _logical(s["v_pages"], s["table"])
    t, i = torch.arange(k.shape[2], device="cuda"), torch.arange(q, device="cuda")
    qn = s["q_lens"] if s["q_lens"] is not None else torch.full_like(s["lens"], q)
    end = ((s["lens"] - qn)[:, None] + i)[..., None]
    seen = (t <= end) & (i < qn[:, None])[..., None]  # [B][q][T]
    x = scores(qf, k).reshape(B, Hkv, G, q, -1).masked_fill_(~seen[:, None, None], -math.inf)
    x = x.reshape(B, Hkv, G * q, -1)
    m = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, Hkv, G, 1).expand(B, -1, -1, q).reshape(B, Hkv, G * q, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - m)
    there = (t < s["lens"][:, None])[:, None, :, None]
    o = torch.matmul(x, v * there)
    # each group over its prefix, all of its rows at once
    starts, lengths = s["starts"].tolist(), s["prefix_lens"].tolist()
    for n in range(s["groups"]):
        a, z, L = starts[n], starts[n + 1], lengths[n]
        if L == 0:
            continue
        kp, vp = (_logical(p, s["prefix_table"][n:n + 1])[0, :, :L] for p in (s["k_pages"], s["v_pages"]))
        x = scores(qf[a:z].transpose(0, 1).reshape(Hkv, (z - a) * G * q, D), kp)
        mp = x.amax(-1, keepdim=True)
        x = x.sub_(mp).exp_()
        lp, op = x.sum(-1, keepdim=True), torch.matmul(x, vp)
        mp, lp, op = (y.reshape(Hkv, z - a, G * q, -1).transpose(0, 1) for y in (mp, lp, op))
        both = torch.maximum(m[a:z], mp)
        old, new = torch.exp(m[a:z] - both), torch.exp(mp - both)
        o[a:z] = o[a:z] * old + op * new
        total[a:z] = total[a:z] * old + lp * new
        m[a:z] = both
    o = (o / total).reshape(B, Hq, q, D)
    lse = (m + torch.log(total)).reshape(B, Hq, q)
    if s["q_lens"] is not None:
        real = (i < qn[:, None])[:, None]
        o, lse = torch.where(real[..., None], o, 0.0), torch.where(real, lse, 0.0)
    return {"out": o.to(s["q_rows"].dtype), "lse": lse}


def _norm_rope(s):
    B, Hkv, n, D = s["k_new"].shape
    rot, half = s["rot"], s["rot"] // 2
    freq = s["theta"] ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / rot))
    angle = s["positions"].double()[..., None] * freq  # [B][n][half]: 64 bits, positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x, w):
        x, w = x.float(), w.float() + s["offset"]
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + s["eps"]) * (w[:, None] if s["per_head"] else w)
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1).to(s["k_pages"].dtype)

    j = torch.arange(n, device="cuda")
    real = torch.ones((B, n), dtype=torch.bool, device="cuda") if s["n_new"] is None else j < s["n_new"][:, None]
    q = torch.where(real[:, None, :, None], turn(s["q"], s["q_weight"]), s["q_out"])
    t = s["past_lens"].long()[:, None] + j
    page = torch.gather(s["table"].long(), 1, torch.where(real, t, 0) // s["P"])[:, None]
    at = (page * Hkv + torch.arange(Hkv, device="cuda")[None, :, None]) * s["P"] + t[:, None] % s["P"]
    use = real[:, None].expand(-1, Hkv, -1)
    s["k_pages"].view(-1, D)[at[use]] = turn(s["k_new"], s["k_weight"])[use]
    s["v_pages"].view(-1, D)[at[use]] = s["v_new"][use]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _resize(s):
    P, table, ring, held, free = s["P"], s["table"], s["ring"], s["n_pages"], s["free"]
    N = ring.numel()
    j = torch.arange(table.shape[1], device="cuda")
    for lens, new, slots in s["steps"]:
        head, count, n, want = free[0].long(), free[1].long(), held.long(), (lens.long() + P - 1) // P
        need = (want - n).clamp(min=0)
        upto = torch.cumsum(need, 0)
        served = upto <= count
        need = torch.where(served, need, 0)
        back = (n - want).clamp(min=0)
        behind = torch.cumsum(back, 0)
        # pages given back go behind the ring's last, those taken come from its front
        given = (j >= want[:, None]) & (j < n[:, None])
        at = (head + count + (behind - back)[:, None] + j - want[:, None]) % N
        taken = (j >= n[:, None]) & (j < (n + need)[:, None])
        source = (head + (upto - need)[:, None] + j - n[:, None]) % N
        fresh = ring[source]
        ring[at[given]] = table[given]
        table.copy_(torch.where(taken, fresh, torch.where(given, -1, table)))
        held.copy_(n + need - back)
        took = need.sum()
        free.copy_(torch.stack([(head + took) % N, count - took + back.sum()]))
        if new is not None:
            i = torch.arange(slots.shape[1], device="cuda")
            t = (lens - new)[:, None] + i
            use = (i < new[:, None]) & served[:, None]
            page = torch.gather(table, 1, torch.where(use, t // P, 0))
            slots.copy_(torch.where(use, page * P + t % P, -1))
    return _resized(s)


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and head at a time."""
    if case["op"] == "resize":
        return None  # whole numbers alone
    s = prepare(case, seed)
    B, Hkv, D, P = s["B"], s["Hkv"], s["D"], s["P"]
    G = s["Hq"] // Hkv
    table = s["table"].tolist()
    if s["op"] == "norm_rope":
        rot, pairs = s["rot"], s["rot"] // 2
        k2, v2, q2 = s["k_pages"].double(), s["v_pages"].double(), s["q_out"].double()
        take = [(2 * p, 2 * p + 1) if s["interleaved"] else (p, p + pairs) for p in range(pairs)]
        first, second = (torch.tensor(x, device="cuda") for x in zip(*take))
        for b in range(B):
            n = s["n"] if s["n_new"] is None else int(s["n_new"][b])
            z = torch.stack([s["positions"][b, :n].double() * s["theta"] ** (-2.0 * p / rot)
                             for p in range(pairs)], -1)
            t = int(s["past_lens"][b]) + np.arange(n)
            page = torch.from_numpy(np.array(table[b])[t // P]).cuda()
            slot = torch.from_numpy(t % P).cuda()
            for src, weight, H in ((s["q"], s["q_weight"], s["Hq"]), (s["k_new"], s["k_weight"], Hkv)):
                for h in range(H):
                    x = src[b, h, :n].double()
                    x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + s["eps"])
                    x = x * ((weight[h] if s["per_head"] else weight).double() + s["offset"])
                    y = x.clone()
                    y[:, first] = x[:, first] * torch.cos(z) - x[:, second] * torch.sin(z)
                    y[:, second] = x[:, first] * torch.sin(z) + x[:, second] * torch.cos(z)
                    if src is s["q"]:
                        q2[b, h, :n] = y
                    else:
                        k2[page, h, slot], v2[page, h, slot] = y, s["v_new"][b, h, :n].double()
        return {"q": q2, "k_pages": k2, "v_pages": v2}

    def rows(pages, ids, h, L):
        at = torch.tensor(ids[: -(-L // P)], dtype=torch.long, device="cuda")
        return pages[at, h].reshape(-1, D)[:L].double()

    q, lens, starts = s["q"], s["lens"].tolist(), s["starts"].tolist()
    counts = [q] * B if s["q_lens"] is None else s["q_lens"].tolist()
    prefix_table, prefix_lens = s["prefix_table"].tolist(), s["prefix_lens"].tolist()
    out = torch.zeros((B, s["Hq"], q, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, s["Hq"], q), dtype=torch.float64, device="cuda")
    for n in range(s["groups"]):
        for h in range(Hkv):
            kp, vp = (rows(p, prefix_table[n], h, prefix_lens[n]) for p in (s["k_pages"], s["v_pages"]))
            for b in range(starts[n], starts[n + 1]):
                L, c = lens[b], counts[b]
                k = torch.cat([kp, rows(s["k_pages"], table[b], h, L)])
                v = torch.cat([vp, rows(s["v_pages"], table[b], h, L)])
                x = (s["q_rows"][b, h * G:(h + 1) * G, :c].double() @ k.T) * s["scale"]
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                pos = torch.arange(L - c, L, device="cuda")[:, None] + prefix_lens[n]
                x = x.masked_fill(torch.arange(k.shape[0], device="cuda") > pos, -math.inf)
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"][h * G:(h + 1) * G].double()[:, None, None].expand(-1, c, 1)], -1)
                lse[b, h * G:(h + 1) * G, :c] = torch.logsumexp(x, -1)
                out[b, h * G:(h + 1) * G, :c] = torch.softmax(x, -1)[..., : k.shape[0]] @ v
    return {"out": out, "lse": lse}
