"""The rotary append with norms (atlas_kv_append_norm_rope) against a plain fp64 form.

Tolerance.  The sum of a row's squares is a chain of at most 16 fused steps and 5 additions of
positive terms, and eps one more: 22 * 2^-24 of it, half of that in its root; rsqrtf is within 2
ulp, 2^-22; the weight's offset and the two products round by 2^-24 each.  Together 18 * 2^-24
of a normed element.  The rotation adds what tests/test_rope_append.py derives, 2^-19 (|x| +
|y|) of a pair's normed elements: below 2^-18 (|x| + |y|) in all, before the store's half step
(2^-8 in bf16; the fp32 store rounds nothing further)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.operator_refs import angle, pair_elements, turned, widen
from tests.serving_refs import normed

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def rope(**kw):
    R = atlas._Rope()
    R.batch, R.max_pages_per_seq, R.num_pages, R.max_new, R.kv_dtype = 2, 4, 8, 0, 1
    R.n_q_heads, R.q, R.q_out, R.positions = 8, 0x1000, 0x2000, 0x3000
    R.n_axes, R.rot_dim, R.theta = 1, 128, 1e4
    for k, v in kw.items():
        setattr(R, k, v)
    return R


def norm(**kw):
    N = atlas._Norm(0x1000, 0x1000, 1, 0, 0.0, 1e-6)
    for k, v in kw.items():
        setattr(N, k, v)
    return N


def call(lib, R, N, ptrs=(0x1000,) * 6):
    return lib.atlas_kv_append_norm_rope(*ptrs, None, 2, 128, 16, ctypes.byref(R) if R else None,
                                         ctypes.byref(N) if N else None)


@pytest.mark.parametrize("kw,status", [
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(per_head=2), 1),
    (dict(per_head=-1), 1), (dict(weight_offset=math.inf), 1), (dict(weight_offset=math.nan), 1),
    (dict(q_weight=0x1008), 1), (dict(k_weight=0x1004), 1), (dict(weight_dtype=2), 2),
    (dict(weight_dtype=-1), 2), ({}, 0), (dict(q_weight=None, k_weight=None, weight_dtype=0), 0),
    (dict(eps=0.0, per_head=1, weight_offset=-1.0), 0)])
def test_refusals(lib, kw, status):
    """(max_new 0: a good call has nothing to do)"""
    assert call(lib, rope(), norm(**kw)) == status


def test_refuses_what_the_call_without_norms_does(lib):
    assert call(lib, None, norm()) == 1 and call(lib, rope(), None) == 1
    assert call(lib, rope(kv_dtype=0), norm(weight_dtype=1)) == 2        # bf16 weights of an fp32 cache
    for kw, status in ((dict(batch=0), 1), (dict(max_new=-1), 1), (dict(rot_dim=31), 1), (dict(theta=0.0), 1),
                       (dict(q=None), 1), (dict(q_out=0x2008), 1), (dict(kv_dtype=2), 2), (dict(n_axes=5), 1)):
        assert call(lib, rope(**kw), norm()) == status
    assert call(lib, rope(), norm(), (None,) + (0x1000,) * 5) == 1


def test_the_plain_form_on_a_case_worked_by_hand():
    # squares 9, 16, 0, 0: mean 6.25, root 2.5
    x = np.array([3.0, 4.0, 0.0, 0.0])
    assert np.allclose(normed(x, np.array([1.0, 2.0, 3.0, 4.0]), 0.0, 0.0), [1.2, 3.2, 0, 0])
    assert np.allclose(normed(x, np.zeros(4), 0.0, 1.0), [1.2, 1.6, 0, 0])
    assert np.allclose(normed(x, np.ones(4), 18.75, 0.0), [0.6, 0.8, 0, 0])


# ------------------------------------------------------------------ on the GPU
def step(dtype, B, Hq, Hkv, D, P, n, past, axes, seed, fused=False, size=1.0):
    r = np.random.default_rng(seed)

    def rows(H):
        x = r.standard_normal((B, H, n, D), dtype=np.float32) * np.float32(size)
        return torch.from_numpy(x).to(DT[dtype]).cuda()

    if fused:
        qkv = torch.cat([rows(Hq), rows(Hkv), rows(Hkv)], 1).transpose(1, 2).contiguous().transpose(1, 2)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    width = max(-(-(x + n) // P) for x in past)
    num = B * width + 3
    table = torch.from_numpy(r.permutation(num)[: B * width].reshape(B, width).astype(np.int32)).cuda()
    pools = [torch.from_numpy(r.standard_normal((num, Hkv, P, D), dtype=np.float32)).to(DT[dtype]).cuda()
             for _ in range(2)]
    pos = torch.from_numpy(r.integers(-3, 2000, (axes, B, n)).astype(np.int32)).cuda()
    return q, k, v, *pools, table, torch.tensor(past, dtype=torch.int32, device="cuda"), pos


def weights(r, heads, D, per_head, kind):
    return torch.from_numpy(r.uniform(0.3, 1.7, (heads, D) if per_head else D).astype(np.float32)).to(kind).cuda()


def expected(q, k, v, kp, vp, table, past, pos, freq, pair_axis, inter, counts, wq, wk, eps, offset):
    """fp64 q_out (NaN where not written) and pools, and the bound |x| + |y| of each element."""
    P = kp.shape[2]
    out = [np.full(q.shape, np.nan), widen(kp), widen(vp)]
    tol = [np.zeros(q.shape), np.zeros(kp.shape)]
    pos = pos.cpu().numpy()
    first, second = pair_elements(len(freq), inter)
    for b in range(k.shape[0]):
        for j in range(counts[b]):
            z = np.array([angle(pos[pair_axis[p], b, j], freq[p]) for p in range(len(freq))])
            t = int(past[b]) + j
            page = int(table[b, t // P])
            for i, at, rows, w in ((0, (b, slice(None), j), q, wq), (1, (page, slice(None), t % P), k, wk)):
                x = normed(widen(rows[b, :, j]), 1.0 if w is None else widen(w), eps,
                           0.0 if w is None else offset)
                out[i][at] = turned(x, z, inter)
                both = np.abs(x)
                both[..., first] += np.abs(x[..., second])
                both[..., second] = both[..., first]
                tol[i][at] = both
            out[2][page, :, t % P] = widen(v[b, :, j])
    return out, tol


CASES = [
    # dtype, B, Hq, Hkv, D, P, n, past, axes, rot, interleaved, fused, counts, options
    ("bf16", 2, 4, 2, 128, 16, 1, [5, 16], 1, 128, False, False, None, {}),
    ("bf16", 3, 8, 2, 128, 16, 37, [0, 15, 100], 3, 128, False, True, None, dict(kind="f32")),
    ("f32", 2, 4, 1, 64, 8, 20, [3, 9], 2, 64, False, False, [20, 7], dict(per_head=True)),
    ("f32", 2, 4, 4, 64, 32, 9, [3, 0], 2, 32, True, True, [0, 9], dict(offset=1.0)),
    ("bf16", 1, 3, 1, 64, 64, 50, [77], 4, 24, False, True, None, dict(per_head=True, offset=1.0)),
    ("bf16", 2, 2, 2, 64, 128, 11, [1, 2], 1, 60, True, False, None, dict(eps=0.0)),   # 2 pairs at a time
    ("f32", 1, 2, 1, 128, 16, 5, [0], 1, 126, False, False, None, {}),                 # 63 pairs: rows by warps
    ("bf16", 2, 3, 1, 128, 16, 5, [0, 4], 2, 6, True, True, [5, 2], dict(per_head=True)),
    ("f32", 2, 2, 1, 64, 16, 3, [7, 0], 1, 2, False, False, [3, 0], dict(kind="f32", offset=1.0)),
    ("bf16", 1, 5, 1, 64, 16, 70, [9], 1, 62, False, True, None, dict(kind="f32", weights=False)),
    ("f32", 2, 8, 2, 128, 64, 33, [100, 4], 3, 128, True, False, None, dict(weights=False, eps=0.25)),
    ("bf16", 2, 8, 2, 128, 64, 70, [100, 4], 3, 96, True, True, None, dict(eps=1e-5)),
    ("bf16", 2, 4, 2, 128, 16, 3, [5, 16], 1, 64, False, False, None, dict(size=1e-4, eps=0.0)),
    ("f32", 2, 4, 2, 128, 16, 5, [3, 30], 1, 10, False, True, None, dict(per_head=True, offset=1.0)),
    ("f32", 1, 2, 1, 128, 16, 3, [3], 1, 70, True, False, None, dict(per_head=True)),
    ("bf16", 1, 2, 2, 64, 16, 3, [3], 1, 36, False, False, None, {}),   # both halves have a rotated part
    ("bf16", 1, 2, 2, 64, 16, 3, [3], 1, 34, True, False, None, dict(per_head=True, kind="f32")),
]


@gpu
@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,P,n,past,axes,rot,inter,fused,counts,opt", CASES)
def test_matches_the_plain_form(dtype, B, Hq, Hkv, D, P, n, past, axes, rot, inter, fused, counts, opt):
    q, k, v, kp, vp, table, lens, pos = step(dtype, B, Hq, Hkv, D, P, n, past, axes, 5 + n, fused,
                                             opt.get("size", 1.0))
    r = np.random.default_rng(77)
    kind = DT[opt.get("kind", dtype)]
    wq, wk = (weights(r, H, D, opt.get("per_head"), kind) if opt.get("weights", True) else None for H in (Hq, Hkv))
    eps, offset = opt.get("eps", 1e-6), opt.get("offset", 0.0)
    pair_axis = tuple(p % axes for p in range(rot // 2))
    freq = [1e6 ** (-2.0 * p / rot) for p in range(rot // 2)]
    (want_q, want_k, want_v), tol = expected(q, k, v, kp, vp, table, past, pos, freq, pair_axis, inter,
                                             counts or [n] * B, wq, wk, eps, offset)
    before = kp.clone(), vp.clone()
    q_out = torch.full((B, Hq, n, D), 99.0, dtype=DT[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=wq, k_weight=wk, eps=eps, weight_offset=offset, theta=1e6, rot_dim=rot,
              pair_axis=pair_axis, interleaved=inter, n_new=None if counts is None else
              torch.tensor(counts, dtype=torch.int32, device="cuda"))
    got = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_out=q_out, status=status, **kw)
    assert got is q_out and int(status.item()) == 0
    store = 2.0 ** -8 if dtype == "bf16" else 0.0
    real = ~np.isnan(want_q)
    assert (widen(q_out)[~real] == 99).all()                  # rows past n_new[b] stay
    for x, y, z in ((widen(q_out)[real], want_q[real], tol[0][real]), (widen(kp), want_k, tol[1])):
        assert (np.abs(x - y) <= 2.0 ** -18 * z + store * np.abs(y)).all()
    assert np.array_equal(widen(vp), want_v)
    # the same queries normed in place, and the same call without queries
    if q.is_contiguous():
        atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_out=q, **kw)
        assert np.array_equal(widen(q)[real], widen(q_out)[real])
    kp2, vp2 = before
    assert atlas.kv_append_norm_rope(None, k, v, kp2, vp2, table, lens, pos, **kw) is None
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)


@gpu
@pytest.mark.parametrize("rot", [128, 126])
@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (3e38, 0.0), (1e-30, 0.0), (1e-37, 0.0), (1e-30, 1e-6)])
def test_squares_that_fp32_does_not_hold(size, eps, rot):
    q, k, v, kp, vp, table, lens, pos = step("f32", 2, 2, 1, 128, 16, 3, [5, 16], 1, 3, size=1.0)
    q, k = (torch.from_numpy((widen(x) / np.abs(widen(x)).max() * size).astype(np.float32)).cuda() for x in (q, k))
    out = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, torch.zeros_like(pos), eps=eps, rot_dim=rot)
    want = normed(widen(q), 1.0, eps, 0.0)
    assert (np.abs(widen(out) - want) <= 2.0 ** -18 * np.abs(want) + 2.0 ** -149).all()


@gpu
@pytest.mark.parametrize("rot", [128, 126])
def test_zeros_infinities_and_nan_stay_in_their_row(rot):
    q, k, v, kp, vp, table, lens, pos = step("f32", 1, 5, 1, 128, 16, 1, [5], 1, 3)
    good = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, rot_dim=rot)
    q = q.clone()
    q[0, 1] = 0.0
    q[0, 2, 0, 7] = float("nan")
    q[0, 3, 0, 100] = float("inf")
    out = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, rot_dim=rot)
    assert torch.equal(out[0, 0], good[0, 0]) and torch.equal(out[0, 4], good[0, 4])
    assert (out[0, 1] == 0).all() and torch.isnan(out[0, 2]).all()
    assert torch.isnan(out[0, 3]).any() and not torch.isinf(out[0, 3]).any()
    out = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, rot_dim=rot, eps=0.0)
    assert torch.isnan(out[0, 1]).all()                         # 0 / 0


@gpu
@pytest.mark.parametrize("rot", [64, 62])
def test_bad_pages_and_lengths_are_reported_and_skipped(rot):
    q, k, v, kp, vp, table, lens, pos = step("bf16", 3, 4, 2, 64, 16, 3, [5, 16, 30], 1, 8)
    good_q = atlas.kv_append_norm_rope(q, k, v, kp.clone(), vp.clone(), table, lens, pos, rot_dim=rot)
    for change, bit in ((("table", (1, 1), -1), 1), (("table", (1, 1), kp.shape[0]), 1),
                        (("lens", 1, -1), 2), (("lens", 1, table.shape[1] * 16 - 2), 2), (("n_new", 1, 4), 2)):
        x = dict(table=table.clone(), lens=lens.clone(), n_new=torch.full_like(lens, 3))
        x[change[0]][change[1]] = change[2]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        a, b = kp.clone(), vp.clone()
        out = torch.full_like(good_q, 7.0)
        atlas.kv_append_norm_rope(q, k, v, a, b, x["table"], x["lens"], pos, n_new=x["n_new"], q_out=out,
                                  rot_dim=rot, status=status)
        assert int(status.item()) == bit
        assert torch.equal(out[0], good_q[0]) and torch.equal(out[2], good_q[2])
        # (n_new out of range skips the sequence, else its queries are written all the same)
        assert (out[1] == 7).all() if change[0] == "n_new" else torch.equal(out[1], good_q[1])


@gpu
@pytest.mark.parametrize("rot", [128, 62])
@pytest.mark.parametrize("per_head", [False, True])
def test_captured_and_replayed_with_other_lengths(rot, per_head):
    q, k, v, kp, vp, table, lens, pos = step("bf16", 3, 4, 2, 128, 16, 5, [5, 16, 30], 1, 8)
    r = np.random.default_rng(4)
    wq, wk = (weights(r, H, 128, per_head, torch.bfloat16) for H in (4, 2))
    counts = torch.full_like(lens, 5)
    kw = dict(q_weight=wq, k_weight=wk, rot_dim=rot, n_new=counts)
    out = torch.zeros_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_out=out, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_out=out, **kw)
    for past, n in (([5, 16, 30], [5, 5, 5]), ([0, 2, 9], [1, 5, 0]), ([40, 42, 15], [5, 1, 3])):
        torch.cuda.synchronize()
        pools = []
        for _ in range(2):
            for t in (kp, vp, out):
                t.fill_(1.0)
            lens.copy_(torch.tensor(past, dtype=torch.int32))
            counts.copy_(torch.tensor(n, dtype=torch.int32))
            if not pools:
                graph.replay()
            else:
                atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_out=out, **kw)
            torch.cuda.synchronize()
            pools.append([t.clone() for t in (kp, vp, out)])
        assert all(torch.equal(a, b) for a, b in zip(*pools))
        assert not (pools[0][0] == 1).all()


@gpu
@pytest.mark.parametrize("rot", [128, 62])
def test_pages_whose_offsets_pass_32_bits(rot):
    q, k, v, kp, vp, table, lens, pos = step("bf16", 3, 4, 2, 128, 128, 5, [5, 16, 200], 1, 8)
    n = kp.shape[0]
    num = (1 << 32) // (2 * 128 * 128) + 2 * n
    far = [torch.empty((num, *kp.shape[1:]), dtype=kp.dtype, device="cuda") for _ in range(2)]
    for a, b in zip(far, (kp, vp)):
        a[num - n:] = b
    a = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, rot_dim=rot)
    b = atlas.kv_append_norm_rope(q, k, v, *far, table + (num - n), lens, pos, rot_dim=rot)
    assert torch.equal(a, b)
    assert torch.equal(far[0][num - n:], kp) and torch.equal(far[1][num - n:], vp)


@gpu
@pytest.mark.parametrize("per_head,rot", [(False, 128), (True, 128), (False, 62)])
def test_many_tokens_are_as_one_by_one(per_head, rot):
    """Two or four tokens a CTA, and the last CTA with fewer: the bits of calls of one token."""
    B, n = 3, 1701
    q, k, v, kp, vp, table, lens, pos = step("bf16", B, 4, 2, 128, 16, n, [5, 16, 30], 1, 8)
    r = np.random.default_rng(4)
    wq, wk = (weights(r, H, 128, per_head, torch.float32) for H in (4, 2))
    kw = dict(q_weight=wq, k_weight=wk, rot_dim=rot)
    pools = kp.clone(), vp.clone()
    out = atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, **kw)
    for i in (0, 1, 450, n - 2, n - 1):
        one = atlas.kv_append_norm_rope(*(t[:, :, i:i + 1] for t in (q, k, v)), *pools, table, lens + i,
                                        pos[:, :, i:i + 1].contiguous(), **kw)
        assert torch.equal(one, out[:, :, i:i + 1])
        for b in range(B):
            t = int(lens[b]) + i
            page = int(table[b, t // 16])
            for x, y in zip(pools, (kp, vp)):
                assert torch.equal(x[page, :, t % 16], y[page, :, t % 16])


def apart(t):
    return torch.stack([t, t], -1)[..., 0]


@gpu
@pytest.mark.parametrize("qw,kw", [
    (lambda t: t.cpu(), None), (lambda t: t.half(), None), (lambda t: t[:32].contiguous(), None), (apart, None),
    (lambda t: t[None], None), (lambda t: t.expand(4, -1).contiguous(), None), (None, lambda t: t.float()),
    (lambda t: t.expand(2, -1).contiguous(), lambda t: t.expand(2, -1).contiguous())])
def test_wrong_weights(qw, kw):
    q, k, v, kp, vp, table, lens, pos = step("bf16", 2, 4, 2, 64, 16, 1, [5, 16], 1, 8)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    before = kp.clone()
    with pytest.raises(ValueError):
        atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos, q_weight=qw(w) if qw else w,
                                  k_weight=kw(w) if kw else w)
    with pytest.raises(atlas.AtlasError):                       # 2 bytes past a 16-byte boundary
        atlas.kv_append_norm_rope(q, k, v, kp, vp, table, lens, pos,
                                  q_weight=torch.ones(65, dtype=torch.bfloat16, device="cuda")[1:])
    torch.cuda.synchronize()
    assert torch.equal(kp, before)
