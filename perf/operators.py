"""The cache operators around the paged attention, as measured work: what a case is, its
inputs, one pass through it, and what that pass has to read, write and compute.

Four operators over the page pools [num_pages][Hkv][P][D] of the library:

  rope     rotary positions with several axes (time, height, width) applied to a step's
           queries and keys while the keys and values go into their pages;
  cross    attention of decoder rows to an encoder's states, held in pages of their own:
           every row sees all of its sequence's encoder states, of which there may be none;
  weights  the attention weight each cached key received from the given query rows, added
           to a running total per (sequence, kv head, key);
  evict    the keys that stay under a budget, picked by that total, and the pages with only
           those keys left in them.

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
        # one sequence's decode step against a short clip's encoder states (latency)
        dict(name="cross_step_f32", op="cross", dtype="f32", B=1, Hq=4, Hkv=4, D=64, P=16, q=1,
             lo=512, hi=512, lens_seed=1, empty=False, ragged=False, sinks=False),
        # a serving batch's decode step, encoder lengths of all sizes, one request without any
        dict(name="cross_step_batch", op="cross", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=16,
             q=1, lo=1, hi=16384, lens_seed=2, empty=True, ragged=False, sinks=False),
        # prompts of a batch, of different lengths, against long encoder states
        dict(name="cross_prompt", op="cross", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, P=64,
             q=1500, lo=3000, hi=8192, lens_seed=3, empty=False, ragged=True, sinks=False),
        # a decode step: one token per sequence, written and rotated
        dict(name="rope_step", op="rope", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=16, n=1,
             past=4000, axes=3, rot=128, interleaved=False, fused=True, ragged=False,
             theta=1000000.0, far=0),
        # an image prompt in fp32: a part of the head rotated, pairs side by side
        dict(name="rope_image_f32", op="rope", dtype="f32", B=2, Hq=16, Hkv=4, D=64, P=32, n=777,
             past=13, axes=2, rot=32, interleaved=True, fused=False, ragged=True, theta=10000.0,
             far=0),
        # long video prompts straight from the fused projection, at far positions
        dict(name="rope_video", op="rope", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, P=64, n=8192,
             past=0, axes=3, rot=128, interleaved=False, fused=True, ragged=False,
             theta=1000000.0, far=400000),
        # totals kept up at each decode step of a batch
        dict(name="weights_step", op="weights", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=16,
             q=1, lo=1024, hi=32768, lens_seed=4, ragged=False, window=0, softcap=0.0),
        # the last rows of long prompts as observers
        dict(name="weights_suffix", op="weights", dtype="bf16", B=8, Hq=64, Hkv=8, D=128, P=64,
             q=32, lo=8192, hi=65536, lens_seed=5, ragged=True, window=0, softcap=0.0),
        # every row of a prompt observes
        dict(name="weights_prompt", op="weights", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, P=64,
             q=8192, lo=8192, hi=8192, lens_seed=6, ragged=False, window=0, softcap=0.0),
        # one short sequence cut a little, in its own pages (latency)
        dict(name="evict_short_f32", op="evict", dtype="f32", B=1, Hkv=4, D=64, P=16, lo=600,
             hi=600, lens_seed=7, budget=512, first=4, recent=64, in_place=True),
        # prompts of a batch cut to an eighth, into fresh pages (their own may be shared)
        dict(name="evict_prompts", op="evict", dtype="bf16", B=8, Hkv=8, D=128, P=16, lo=1000,
             hi=32768, lens_seed=8, budget=4096, first=4, recent=512, in_place=False),
        # one very long sequence halved in its own pages
        dict(name="evict_long", op="evict", dtype="bf16", B=1, Hkv=8, D=128, P=64, lo=131072,
             hi=131072, lens_seed=9, budget=65536, first=16, recent=4096, in_place=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the listed ranges.  One that would need more than its operator's
    largest listed case gets a smaller batch, then shorter sequences."""
    op = rng.choice(["cross", "rope", "weights", "evict"])
    D = rng.choice([64, 128])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log_int(rng, 1, 32),
             Hkv=rng.choice([1, 2, 4, 8]), D=D, P=rng.choice([8, 16, 32, 64, 128]))
    G = rng.choice([1, 2, 3, 4, 8])
    hi = _log_int(rng, 100, 32768)
    if op == "cross":
        c.update(Hq=c["Hkv"] * G, q=rng.choice([1, 1, _log_int(rng, 2, 1500)]),
                 lo=rng.choice([1, hi // 2 + 1]), hi=hi, lens_seed=rng.randrange(1 << 20),
                 empty=rng.random() < 0.4, ragged=rng.random() < 0.4, sinks=rng.random() < 0.3)
    elif op == "rope":
        inter = rng.random() < 0.4
        c.update(Hq=c["Hkv"] * G, n=rng.choice([1, _log_int(rng, 2, 8192)]),
                 past=rng.randrange(0, 3000), axes=rng.choice([1, 2, 3, 4]),
                 rot=rng.choice([D, D, D // 2, 24]), interleaved=inter,
                 fused=rng.random() < 0.5, ragged=rng.random() < 0.4,
                 theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                 far=rng.choice([0, 0, _log_int(rng, 1000, 1000000)]))
    elif op == "weights":
        q = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 65, 8192)])
        hi = max(hi, q)
        c.update(Hq=c["Hkv"] * G, q=q, lo=rng.choice([q, max(q, hi // 2)]), hi=hi,
                 lens_seed=rng.randrange(1 << 20), ragged=rng.random() < 0.4,
                 window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]),
                 softcap=rng.choice([0.0, 0.0, 0.0, 30.0]))
    else:
        budget = _log_int(rng, 16, hi)
        first = min(rng.choice([0, 4, 16]), budget)
        c.update(lo=rng.choice([1, hi // 2 + 1]), hi=hi, lens_seed=rng.randrange(1 << 20),
                 budget=budget, first=first, recent=rng.randrange(0, (budget - first) // 2 + 1),
                 in_place=rng.random() < 0.5)
    most = {k: max(work(x)[k] for x in listed() if x["op"] == op) for k in ("bytes", "flops")}
    while any(work(c)[k] > most[k] for k in most):
        if c["B"] > 1:
            c["B"] = c["B"] // 2
        elif c.get("n", 0) > 1:
            c["n"] //= 2
        elif c.get("q", 0) > 64:
            c["q"] //= 2
        else:
            c["hi"] = max(c["hi"] // 2, c.get("q", 1))
            c["lo"] = min(c["lo"], c["hi"])
    return c


def _lens(c):
    """Key lengths of the sequences: a pure function of the case."""
    r = random.Random(c["lens_seed"])
    lens = np.array([r.randint(c["lo"], c["hi"]) for _ in range(c["B"])])
    lens[0] = c["hi"]
    if c.get("empty") and c["B"] > 1:
        lens[1] = 0
    return lens


def _rows(c, n):
    """Rows of each sequence: n, or up to n (the last sequence short) in a ragged batch."""
    return np.array([n] + [max(1, n - (b * 37) % n) for b in range(1, c["B"])]) \
        if c["ragged"] else np.full(c["B"], n)


def work(case):
    c = case
    e = _BYTES[c["dtype"]]
    D = c["D"]
    if c["op"] == "rope":
        rows = int(_rows(c, c["n"]).sum())
        moved = 2 * rows * (c["Hq"] + 2 * c["Hkv"]) * D * e
        return {"bytes": moved + 4 * rows * c["axes"], "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    lens = _lens(c)
    if c["op"] == "cross":
        rows = _rows(c, c["q"])
        pairs = c["Hq"] * int((rows * lens).sum())
        return {"bytes": 2 * int(lens.sum()) * c["Hkv"] * D * e + 2 * int(rows.sum()) * c["Hq"] * D * e
                + 4 * int(rows.sum()) * c["Hq"], "flops": pairs * (4 * D + 4)}
    if c["op"] == "weights":
        rows = _rows(c, c["q"])
        if c["window"]:
            seen = np.minimum(lens, c["window"] + rows)
            pairs = int((rows * np.minimum(lens, c["window"])).sum())
        else:
            seen = lens
            pairs = int((rows * lens - rows * (rows - 1) // 2).sum())
        return {"bytes": int(seen.sum()) * c["Hkv"] * (D * e + 8) + int(rows.sum()) * c["Hq"] * (D * e + 4),
                "flops": pairs * c["Hq"] * (2 * D + 4)}
    kept = np.minimum(lens, c["budget"])
    return {"bytes": 4 * int(lens.sum()) * c["Hkv"] + 8 * int(kept.sum()) * c["Hkv"]
            + 4 * int(kept.sum()) * c["Hkv"] * D * e, "flops": int(lens.sum()) * c["Hkv"]}


def _tensor(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, dt = case, _DT[case["dtype"]]
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    s = dict(c)
    if c["op"] == "rope":
        past = np.full(B, c["past"]) + np.arange(B) % 7
        total = past + c["n"]
    else:
        total = _lens(c)
    pages = -(-total // P)
    width = max(1, int(pages.max()))
    fresh = -(-min(c["budget"], int(total.max())) // P) if c["op"] == "evict" and not c["in_place"] else 0
    num = int(pages.sum()) + B * fresh + 3
    # every page belongs to one sequence; what lies behind a sequence's end is stale data
    perm = torch.randperm(num, generator=g, device="cuda", dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(pages)])[:-1]
    at = torch.from_numpy(first[:, None] + np.arange(width)[None]).cuda()
    inside = torch.from_numpy(np.arange(width)[None] < pages[:, None]).cuda()
    s["table"] = torch.where(inside, perm[at.clamp(max=num - 1)], 0).to(torch.int32)
    s["k_pages"] = normal(num, Hkv, P, D)
    if c["op"] != "weights":
        s["v_pages"] = normal(num, Hkv, P, D)
    if c["op"] == "evict":
        s["lens"] = _tensor(total)
        # the totals of real rows: most keys get little, a few most of the weight
        w = torch.empty((B, Hkv, width * P), device="cuda").exponential_(generator=g)
        s["w"] = w.pow_(4.0)
        if fresh:
            base = int(pages.sum())
            s["new_table"] = perm[base:base + B * fresh].reshape(B, fresh).contiguous()
        else:
            s["new_table"] = None
        return s
    if c["op"] == "rope":
        n, Hq = c["n"], c["Hq"]
        if c["fused"]:  # one projection's output, token after token
            qkv = normal(B, n, Hq + 2 * Hkv, D).transpose(1, 2)
            s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = normal(B, Hq, n, D), normal(B, Hkv, n, D), normal(B, Hkv, n, D)
        s["q_out"] = torch.zeros((B, Hq, n, D), dtype=dt, device="cuda")
        s["past_lens"] = _tensor(past)
        s["n_new"] = _tensor(_rows(c, n)) if c["ragged"] else None
        # frames of 24 x 32 patches: time advances once per frame
        j = torch.arange(n, device="cuda")
        grid = torch.stack([j // 768, j // 32 % 24, j % 32, j])[: c["axes"]]
        shift = torch.randint(0, 50, (c["axes"], B, 1), generator=g, device="cuda")
        s["positions"] = (grid[:, None, :] + shift + c["far"]).to(torch.int32).contiguous()
        pairs = c["rot"] // 2
        s["pair_axis"] = tuple(k * c["axes"] // pairs for k in range(pairs))
        s["axis"] = torch.tensor(s["pair_axis"], device="cuda")
        return s
    Hq, q = c["Hq"], c["q"]
    s["lens"] = _tensor(total)
    s["scale"] = 1.0 / math.sqrt(D)
    s["q_rows"] = normal(B, Hq, q, D)
    s["q_lens"] = _tensor(np.minimum(_rows(c, q), total) if c["op"] == "weights" else _rows(c, q)) \
        if c["ragged"] else None
    if c["op"] == "cross":
        s["out"] = torch.zeros((B, Hq, q, D), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((B, Hq, q), device="cuda")
        s["sink"] = torch.randn(Hq, generator=g, device="cuda") if c["sinks"] else None
        return s
    # the row sums that the attention left behind, one kv head of one sequence at a time
    s["w"] = torch.rand((B, Hkv, width * P), generator=g, device="cuda") * (Hq // Hkv * q / int(total.max()))
    lse = torch.empty((B, Hq, q), device="cuda")
    G = Hq // Hkv
    for b in range(B):
        L = int(total[b])
        qn = int(min(_rows(c, q)[b], L))
        pos = torch.arange(q, device="cuda")[:, None] + (L - qn)
        t = torch.arange(L, device="cuda")[None]
        seen = (t <= pos) & (t > pos - c["window"] if c["window"] else t >= 0)
        rows = s["k_pages"][s["table"][b, : -(-L // P)].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        for h in range(Hkv):
            x = torch.matmul(s["q_rows"][b, h * G:(h + 1) * G].float(), rows[h].float().T) * s["scale"]
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x.masked_fill(~seen, -math.inf), -1)
    s["lse"] = lse
    return s


def run(state):
    s = state
    if own:
        return _own(s)
    return {"cross": _cross, "rope": _rope, "weights": _weights, "evict": _evict}[s["op"]](s)


def _own(s):
    import exact_causal_gqa_gb300 as atlas
    if s["op"] == "cross":
        out = atlas.cross(s["q_rows"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["Hq"],
                          s["Hkv"], s["D"], s["P"], s["scale"], out=s["out"], lse=s["lse"],
                          q_lens=s["q_lens"], sinks=s["sink"])
        return {"out": out, "lse": s["lse"]}
    if s["op"] == "rope":
        q = atlas.kv_append_rope(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"],
                                 s["table"], s["past_lens"], s["positions"], theta=s["theta"],
                                 rot_dim=s["rot"], pair_axis=s["pair_axis"],
                                 interleaved=s["interleaved"], n_new=s["n_new"], q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["op"] == "weights":
        return {"w": atlas.kv_weights(s["q_rows"], s["k_pages"], s["table"], s["lens"], s["lse"],
                                      s["Hq"], s["Hkv"], s["D"], s["P"], s["scale"], weights=s["w"],
                                      q_lens=s["q_lens"], window=s["window"], softcap=s["softcap"])}
    kept, lens, w = atlas.kv_select(s["w"], s["lens"], s["budget"], keep_first=s["first"],
                                    keep_recent=s["recent"])
    atlas.kv_compact(s["k_pages"], s["v_pages"], s["table"], kept, lens, new_page_table=s["new_table"])
    return {"kept": kept, "lens": lens, "w": w, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _logical(pages, table):
    """[num_pages][Hkv][P][D] through the table -> [B][Hkv][width * P][D] in fp32."""
    x = pages[table.long()].transpose(1, 2).float()
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _cross(s):
    B, Hq, q, D = s["q_rows"].shape
    k, v = _logical(s["k_pages"], s["table"]), _logical(s["v_pages"], s["table"])
    G = Hq // s["Hkv"]
    there = (torch.arange(k.shape[2], device="cuda") < s["lens"][:, None])[:, None, None]
    x = torch.matmul(s["q_rows"].float().reshape(B, s["Hkv"], G * q, D), k.transpose(2, 3)) * s["scale"]
    x = x.masked_fill(~there, -math.inf)
    m = x.amax(-1, keepdim=True)
    sink = None
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, s["Hkv"], G, 1).expand(B, -1, -1, q).reshape(B, s["Hkv"], G * q, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    o = torch.matmul(x, v * there.transpose(2, 3)) / torch.where(total == 0, 1.0, total)
    o, lse = o.reshape(B, Hq, q, D), (m + torch.log(total)).reshape(B, Hq, q)
    if s["q_lens"] is not None:
        real = (torch.arange(q, device="cuda") < s["q_lens"][:, None])[:, None]
        o, lse = o * real[..., None], torch.where(real, lse, 0.0)
    return {"out": o.to(s["q_rows"].dtype), "lse": lse}


def _slots(table, t, Hkv, P):
    """Rows of the pools seen as [num_pages * Hkv * P][D] that hold keys t [B][Hkv][n]."""
    page = torch.gather(table.long()[:, None].expand(-1, Hkv, -1), 2, t // P)
    return (page * Hkv + torch.arange(Hkv, device="cuda")[None, :, None]) * P + t % P


def _rope(s):
    B, Hkv, n, D = s["k_new"].shape
    rot, half = s["rot"], s["rot"] // 2
    freq = s["theta"] ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / rot))
    angle = s["positions"].double()[s["axis"]].permute(1, 2, 0) * freq  # [B][n][half]: 64 bits, positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        x = x.float()
        if s["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    dt = s["k_pages"].dtype
    j = torch.arange(n, device="cuda")
    real = torch.ones((B, n), dtype=torch.bool, device="cuda") if s["n_new"] is None else j < s["n_new"][:, None]
    q = torch.where(real[:, None, :, None], turn(s["q"]).to(dt), s["q_out"])
    t = (s["past_lens"].long()[:, None] + j)[:, None].expand(-1, Hkv, -1)
    use = real[:, None].expand(-1, Hkv, -1)
    at = _slots(s["table"], torch.where(use, t, 0), Hkv, s["P"])[use]
    s["k_pages"].view(-1, D)[at] = turn(s["k_new"]).to(dt)[use]
    s["v_pages"].view(-1, D)[at] = s["v_new"][use]
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _weights(s):
    B, Hq, q, D = s["q_rows"].shape
    Hkv = s["Hkv"]
    G = Hq // Hkv
    k = _logical(s["k_pages"], s["table"])
    x = torch.matmul(s["q_rows"].float().reshape(B, Hkv, G * q, D), k.transpose(2, 3)) * s["scale"]
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    qn = s["q_lens"] if s["q_lens"] is not None else torch.full_like(s["lens"], q)
    i = torch.arange(q, device="cuda")
    pos = (s["lens"] - qn)[:, None] + i
    t = torch.arange(k.shape[2], device="cuda")
    seen = (t <= pos[..., None]) & (i < qn[:, None])[..., None]
    if s["window"]:
        seen &= t > pos[..., None] - s["window"]
    x = x.reshape(B, Hkv, G, q, -1)
    x.sub_(s["lse"].reshape(B, Hkv, G, q, 1)).masked_fill_(~seen[:, None, None], -math.inf).exp_()
    s["w"].add_(x.sum((2, 3)))
    return {"w": s["w"]}


def _evict(s):
    w, T, Hkv = s["w"], s["w"].shape[-1], s["Hkv"]
    lens, n = s["lens"].long()[:, None, None], s["budget"]
    t = torch.arange(T, device="cuda")[None, None]
    # those that must stay, then the others, then what lies behind the end
    rank = torch.where(t >= lens, 2, torch.where((t < s["first"]) | (t >= lens - s["recent"]), 0, 1))
    order = torch.sort(torch.nan_to_num(w, nan=-math.inf, posinf=math.inf, neginf=-math.inf),
                       dim=-1, descending=True, stable=True).indices
    order = torch.gather(order, -1, torch.sort(torch.gather(rank.expand_as(w), -1, order), dim=-1,
                                               stable=True).indices)
    new = torch.clamp(lens, max=n)
    order = torch.nn.functional.pad(order[..., :n], (0, max(0, n - T)))
    j = torch.arange(n, device="cuda")[None, None]
    kept = torch.sort(torch.where(j < new, order, T), dim=-1).values
    use = (j < new).expand_as(kept)
    kept = torch.where(use, kept, -1)
    kept_w = torch.where(use, torch.gather(w, -1, kept.clamp(min=0)), 0.0)
    src = _slots(s["table"], kept.clamp(min=0), Hkv, s["P"])[use]
    to = s["table"] if s["new_table"] is None else s["new_table"]
    dst = _slots(to, torch.where(use, j, 0), Hkv, s["P"])[use]
    for_k, for_v = s["k_pages"].view(-1, s["D"]), s["v_pages"].view(-1, s["D"])
    for_k[dst], for_v[dst] = for_k[src], for_v[src]
    return {"kept": kept.int(), "lens": new.flatten().int(), "w": kept_w, "k_pages": s["k_pages"],
            "v_pages": s["v_pages"]}


def exact(case, seed):
    """The operators from their definitions in 64 bits, one sequence and kv head at a time."""
    s = prepare(case, seed)
    B, Hkv, D, P = s["B"], s["Hkv"], s["D"], s["P"]
    table = s["table"].tolist()

    def rows(pages, b, h, L):
        return pages[torch.tensor(table[b][: -(-L // P)], dtype=torch.long, device="cuda"), h].reshape(-1, D)[:L].double()

    if s["op"] == "evict":
        kept = np.full((B, Hkv, s["budget"]), -1, np.int32)
        kept_w = np.zeros((B, Hkv, s["budget"]))
        w, lens = s["w"].double().cpu().numpy(), s["lens"].tolist()
        k, v = s["k_pages"], s["v_pages"]
        k2, v2 = k.clone(), v.clone()
        to = table if s["new_table"] is None else s["new_table"].tolist()
        for b in range(B):
            L = lens[b]
            n = min(L, s["budget"])
            for h in range(Hkv):
                must = [t for t in range(L) if t < s["first"] or t >= L - s["recent"]]
                rest = np.setdiff1d(np.arange(L), must)
                rest = rest[np.lexsort((rest, -w[b, h, rest]))]
                got = np.sort(np.concatenate([must, rest])[:n]) if L > n else np.arange(L)
                got = got.astype(np.int64)
                kept[b, h, :n], kept_w[b, h, :n] = got, w[b, h, got]
                a = torch.from_numpy(np.array(table[b])[got // P]).cuda()
                z = torch.from_numpy(np.array(to[b])[np.arange(n) // P]).cuda()
                i, j = torch.from_numpy(got % P).cuda(), torch.arange(n, device="cuda") % P
                k2[z, h, j], v2[z, h, j] = k[a, h, i], v[a, h, i]
        return {"kept": None, "lens": None, "w": torch.from_numpy(kept_w), "k_pages": k2, "v_pages": v2}
    if s["op"] == "rope":
        rot, pairs = s["rot"], s["rot"] // 2
        k2, v2, q2 = s["k_pages"].double(), s["v_pages"].double(), s["q_out"].double()
        take = [(2 * p, 2 * p + 1) if s["interleaved"] else (p, p + pairs) for p in range(pairs)]
        first, second = (torch.tensor(x, device="cuda") for x in zip(*take))
        for b in range(B):
            n = s["n"] if s["n_new"] is None else int(s["n_new"][b])
            z = torch.stack([s["positions"][s["pair_axis"][p], b, :n].double() * s["theta"] ** (-2.0 * p / rot)
                             for p in range(pairs)], -1)
            for src, h, dst in [(s["q"], h, "q") for h in range(s["Hq"])] + [(s["k_new"], h, "k") for h in range(Hkv)]:
                x = src[b, h, :n].double()
                y = x.clone()
                y[:, first] = x[:, first] * torch.cos(z) - x[:, second] * torch.sin(z)
                y[:, second] = x[:, first] * torch.sin(z) + x[:, second] * torch.cos(z)
                if dst == "q":
                    q2[b, h, :n] = y
                    continue
                t = int(s["past_lens"][b]) + np.arange(n)
                page = torch.from_numpy(np.array(table[b])[t // P]).cuda()
                slot = torch.from_numpy(t % P).cuda()
                k2[page, h, slot], v2[page, h, slot] = y, s["v_new"][b, h, :n].double()
        return {"q": q2, "k_pages": k2, "v_pages": v2}
    G, q, lens = s["Hq"] // Hkv, s["q"], s["lens"].tolist()
    counts = [q] * B if s["q_lens"] is None else s["q_lens"].tolist()
    if s["op"] == "cross":
        out = torch.zeros((B, s["Hq"], q, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, s["Hq"], q), dtype=torch.float64, device="cuda")
    else:
        w = s["w"].double()
    for b in range(B):
        L, n = lens[b], counts[b]
        for h in range(Hkv):
            k = rows(s["k_pages"], b, h, L)
            for a in range(h * G, (h + 1) * G):
                x = s["q_rows"][b, a, :n].double() @ k.T * s["scale"]
                if s["op"] == "cross":
                    if s["sink"] is not None:
                        x = torch.cat([x, s["sink"][a].double().expand(n, 1)], 1)
                    lse[b, a, :n] = torch.logsumexp(x, 1) if x.shape[1] else -math.inf
                    if L:
                        out[b, a, :n] = torch.softmax(x, 1)[:, :L] @ rows(s["v_pages"], b, h, L)
                    continue
                if s["softcap"]:
                    x = s["softcap"] * torch.tanh(x / s["softcap"])
                pos = torch.arange(L - n, L, device="cuda")[:, None]
                t = torch.arange(L, device="cuda")[None]
                hidden = (t > pos) | ((t <= pos - s["window"]) if s["window"] else (t < 0))
                x = torch.exp(x - s["lse"][b, a, :n, None].double()).masked_fill(hidden, 0.0)
                w[b, h, :L] += x.sum(0)
    return {"out": out, "lse": lse} if s["op"] == "cross" else {"w": w}
