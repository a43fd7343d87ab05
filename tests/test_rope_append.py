"""The rotary append (atlas_kv_append_rope) against a plain fp64 form.

Tolerance.  The angle is off by at most 2^-24 turns (fixed point; as much again for a
frequency whose last bit another pow rounds differently) and pi/4 2^-24 (its fp32 form),
sincospif by 2 ulp of at most 1: cosine and sine by at most 2 * 2 pi 2^-24 + pi/4 2^-24
+ 2^-23 < 1.0e-6.  The two products and their sum round once each, 3 * 2^-24 of at most
|x| + |y|.  A result is therefore within 2^-19 (|x| + |y|) of the exact one before its
store, which rounds by half a step of the value: 2^-24 in fp32, 2^-8 in bf16; the values
rounded are the computed ones, 1 + 2^-8 of that 2^-19, which the 1.0e-6 leaves room for."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.operator_refs import angle, pair_elements, turned, widen

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def rope(**kw):
    R = atlas._Rope()
    R.batch, R.max_pages_per_seq, R.num_pages, R.max_new, R.kv_dtype = 2, 4, 8, 3, 1
    R.n_q_heads, R.q, R.q_out, R.positions = 8, 0x1000, 0x2000, 0x3000
    R.n_axes, R.rot_dim, R.theta = 3, 128, 1e4
    for k, v in kw.items():
        setattr(R, k, v)
    return R


def call(lib, R, ptrs=(0x1000,) * 6, Hkv=2, D=128, P=16):
    return lib.atlas_kv_append_rope(*ptrs, None, Hkv, D, P, ctypes.byref(R) if R else None)


def i32(*x):
    a = (ctypes.c_int32 * len(x))(*x)
    call.keep = a
    return ctypes.addressof(a)


def f64(*x):
    a = (ctypes.c_double * len(x))(*x)
    call.keep = a
    return ctypes.addressof(a)


@pytest.mark.parametrize("kw,args,status", [
    (dict(batch=0), {}, 1), (dict(max_new=-1), {}, 1), (dict(num_pages=0), {}, 1),
    (dict(n_axes=0), {}, 1), (dict(n_axes=5), {}, 1), (dict(rot_dim=0), {}, 1),
    (dict(rot_dim=31), {}, 1), (dict(rot_dim=130), {}, 1), (dict(interleaved=2), {}, 1),
    (dict(theta=0.0), {}, 1), (dict(theta=-1.0), {}, 1), (dict(theta=math.inf), {}, 1),
    (dict(theta=math.nan), {}, 1), (dict(positions=None), {}, 1), (dict(q=None), {}, 1),
    (dict(q_out=None), {}, 1), (dict(q_out=0x2008), {}, 1), (dict(n_q_heads=-1), {}, 1),
    (dict(n_q_heads=1 << 20), {}, 1), (dict(max_new=1 << 30), {}, 1),
    (dict(kv_dtype=2), {}, 2), ({}, dict(D=96), 2), ({}, dict(P=24), 2), ({}, dict(P=256), 2),
    ({}, dict(Hkv=0), 1), ({}, dict(ptrs=(0x1008,) + (0x1000,) * 5), 1),
    ({}, dict(ptrs=(None,) + (0x1000,) * 5), 1),
])
def test_refusals(lib, kw, args, status):
    assert call(lib, rope(**kw), **args) == status


def test_refuses_bad_host_arrays_and_strides(lib):
    assert call(lib, None) == 1
    assert call(lib, rope(rot_dim=4, pair_axis=i32(0, 3))) == 1       # three axes: 0, 1, 2
    assert call(lib, rope(rot_dim=4, pair_axis=i32(-1, 0))) == 1
    assert call(lib, rope(rot_dim=4, inv_freq=f64(1.0, math.inf))) == 1
    assert call(lib, rope(rot_dim=4, inv_freq=f64(math.nan, 1.0))) == 1
    R = rope()
    R.k_strides = (ctypes.c_int64 * 3)(1024, 128, 132)                # 264 bytes: not 16-byte rows
    assert call(lib, R) == 1
    assert call(lib, rope(max_new=0)) == 0                            # nothing to do, no launch


def test_sections():
    assert atlas.rope_sections((2, 1, 3)) == (0, 0, 1, 2, 2, 2)
    assert atlas.rope_sections((2, 1, 3), cycle=True) == (0, 1, 2, 0, 2, 2)
    assert atlas.rope_sections((0, 2)) == (1, 1)


def test_the_plain_form_on_a_case_worked_by_hand():
    x = np.array([3.0, 4.0, 5.0, 6.0, 7.0])
    z = np.array([math.pi / 2, math.pi])
    assert np.allclose(turned(x, z, False), [-5, -4, 3, -6, 7])
    assert np.allclose(turned(x, z, True), [-4, 3, -5, -6, 7])


# ------------------------------------------------------------------ on the GPU
def step(dtype, B, Hq, Hkv, D, P, n, past, axes, seed, fused=False, far=0, slack=3):
    r = np.random.default_rng(seed)

    def rows(H):
        return torch.from_numpy(r.standard_normal((B, H, n, D), dtype=np.float32)).to(DT[dtype]).cuda()

    if fused:
        qkv = torch.cat([rows(Hq), rows(Hkv), rows(Hkv)], 1).transpose(1, 2).contiguous().transpose(1, 2)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        assert not q.is_contiguous() or n == 1 or Hq == 0
    else:
        q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    width = max(-(-(x + n) // P) for x in past)
    num = B * width + slack
    table = torch.from_numpy(r.permutation(num)[: B * width].reshape(B, width).astype(np.int32)).cuda()
    pools = [torch.from_numpy(r.standard_normal((num, Hkv, P, D), dtype=np.float32)).to(DT[dtype]).cuda()
             for _ in range(2)]
    pos = torch.from_numpy((r.integers(0, 2000, (axes, B, n)) + far).astype(np.int32)).cuda()
    return q, k, v, *pools, table, torch.tensor(past, dtype=torch.int32, device="cuda"), pos


def expected(q, k, v, kp, vp, table, past, pos, freq, pair_axis, interleaved, counts):
    """fp64 q_out (NaN where not written) and pools, and the bound |x| + |y| of each element."""
    P = kp.shape[2]
    out = [np.full(q.shape, np.nan), widen(kp), widen(vp)]
    tol = [np.zeros(q.shape), np.zeros(kp.shape), np.zeros(vp.shape)]
    pos = pos.cpu().numpy()
    first, second = pair_elements(len(freq), interleaved)
    for b in range(k.shape[0]):
        for j in range(counts[b]):
            z = np.array([angle(pos[pair_axis[p], b, j], freq[p]) for p in range(len(freq))])
            t = int(past[b]) + j
            page = int(table[b, t // P])

            def put(i, at, x):
                out[i][at] = turned(x, z, interleaved)
                both = np.abs(x)
                both[..., first] += np.abs(x[..., second])
                both[..., second] = both[..., first]
                tol[i][at] = both

            put(0, (b, slice(None), j), widen(q[b, :, j]))
            put(1, (page, slice(None), t % P), widen(k[b, :, j]))
            out[2][page, :, t % P] = widen(v[b, :, j])
    return out, tol


CASES = [
    # dtype, B, Hq, Hkv, D, P, n, past, axes, rot, interleaved, fused, counts, far
    ("bf16", 2, 4, 2, 128, 16, 1, [5, 16], 3, 128, False, False, None, 0),
    ("bf16", 3, 8, 2, 128, 16, 37, [0, 15, 100], 3, 128, False, True, None, 0),
    ("f32", 2, 4, 1, 64, 8, 20, [3, 9], 2, 64, False, False, [20, 7], 0),
    ("f32", 2, 4, 4, 64, 32, 9, [3, 0], 2, 32, True, True, [0, 9], 0),
    ("bf16", 1, 3, 1, 64, 64, 50, [77], 4, 24, False, True, None, 0),    # 12 pairs: 4 at a time
    ("bf16", 2, 2, 2, 64, 128, 11, [1, 2], 1, 60, True, False, None, 0),  # 30 pairs: 2 at a time
    ("f32", 1, 2, 1, 128, 16, 5, [0], 1, 126, False, False, None, 0),     # 63 pairs: one at a time
    ("bf16", 1, 2, 1, 128, 16, 5, [0], 1, 2, True, True, None, 0),
    ("f32", 2, 8, 2, 128, 64, 33, [100, 4], 3, 128, True, False, None, 10 ** 6),
    ("bf16", 2, 8, 2, 128, 64, 70, [100, 4], 3, 96, True, True, None, 2 ** 31 - 2001),
    ("f32", 1, 4, 1, 64, 16, 12, [0], 2, 64, False, False, None, -(2 ** 31)),
]


@gpu
@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,P,n,past,axes,rot,inter,fused,counts,far", CASES)
def test_matches_the_plain_form(dtype, B, Hq, Hkv, D, P, n, past, axes, rot, inter, fused, counts, far):
    q, k, v, kp, vp, table, lens, pos = step(dtype, B, Hq, Hkv, D, P, n, past, axes, 5 + n, fused, far)
    pair_axis = tuple(p % axes for p in range(rot // 2))
    freq = [1e6 ** (-2.0 * p / rot) for p in range(rot // 2)]
    (want_q, want_k, want_v), tol = expected(q, k, v, kp, vp, table, past, pos, freq, pair_axis,
                                             inter, counts or [n] * B)
    before = kp.clone(), vp.clone()
    q_out = torch.full((B, Hq, n, D), 99.0, dtype=DT[dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(rot_dim=rot, pair_axis=pair_axis, interleaved=inter, n_new=None if counts is None else
              torch.tensor(counts, dtype=torch.int32, device="cuda"))
    got = atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos, theta=1e6, q_out=q_out,
                               status=status, **kw)
    assert got is q_out and int(status.item()) == 0
    store = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    real = ~np.isnan(want_q)
    assert (widen(q_out)[~real] == 99).all()                  # rows past n_new[b] stay
    for x, y, z in ((widen(q_out)[real], want_q[real], tol[0][real]), (widen(kp), want_k, tol[1])):
        assert (np.abs(x - y) <= 2.0 ** -19 * z + store * np.abs(y)).all()
    assert np.array_equal(widen(vp), want_v)
    untouched = tol[1] == 0
    assert np.array_equal(widen(kp)[untouched], widen(before[0])[untouched])
    if inter or rot < D:                                        # the copied elements, bit for bit
        assert np.array_equal(widen(q_out)[..., rot:][real[..., rot:]], widen(q)[..., rot:][real[..., rot:]])
    # the same queries rotated in place, and the same call without queries
    if q.is_contiguous():
        atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos, theta=1e6, q_out=q, **kw)
        assert np.array_equal(widen(q)[real], widen(q_out)[real])
    kp2, vp2 = before
    assert atlas.kv_append_rope(None, k, v, kp2, vp2, table, lens, pos, inv_freq=freq, **kw) is None
    assert torch.equal(kp2, kp) and torch.equal(vp2, vp)


@gpu
def test_position_zero_is_the_plain_append():
    q, k, v, kp, vp, table, lens, pos = step("bf16", 2, 4, 2, 128, 16, 9, [3, 40], 3, 1)
    kp2, vp2 = kp.clone(), vp.clone()
    got = atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos * 0)
    atlas.kv_append(k, v, kp2, vp2, table, lens)
    assert torch.equal(got, q) and torch.equal(kp, kp2) and torch.equal(vp, vp2)


@gpu
def test_scores_depend_on_the_difference_of_positions():
    """<turn(q, a), turn(k, b)> is a function of a - b: the same at 0 and a million on."""
    q, k, v, kp, vp, table, lens, pos = step("f32", 1, 2, 2, 64, 16, 8, [0], 1, 2)
    dots = []
    for shift in (0, 10 ** 6, -(10 ** 9)):
        a = atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos + shift)
        logical = kp[table[0].long()].transpose(0, 1).reshape(2, -1, 64)[:, :8]
        dots.append(a[0].double() @ logical.double().transpose(1, 2))
    norm = (q.double().norm(dim=-1)[0][..., None] * k.double().norm(dim=-1)[0][:, None])
    # each rotated element is off by 2^-19 (|x| + |y|): a row by 2^-18 of its norm at
    # most, a dot of two such rows by 2 * 2^-18 |q| |k|, and two dots are compared
    for d in dots[1:]:
        assert ((d - dots[0]).abs() <= 4 * 2.0 ** -18 * norm).all()


@gpu
def test_bad_pages_lengths_and_counts_are_reported():
    q, k, v, kp, vp, table, lens, pos = step("bf16", 3, 4, 2, 128, 16, 6, [12, 12, 12], 2, 3)
    clean_k, clean_v = kp.clone(), vp.clone()
    good = atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos)
    want_k, want_v = kp, vp

    def run(table=table, lens=lens, n_new=None):
        kk, vv = clean_k.clone(), clean_v.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(good, 99.0)
        atlas.kv_append_rope(q, k, v, kk, vv, table, lens, pos, status=status, q_out=out, n_new=n_new)
        return int(status.item()), out, kk, vv

    bad = table.clone()
    bad[1, 1] = kp.shape[0]
    status, out, kk, vv = run(table=bad)
    assert status == atlas.DEV_BAD_PAGE and torch.equal(out, good)
    page = int(table[1, 1])
    assert torch.equal(kk[page], clean_k[page]) and torch.equal(vv[page], clean_v[page])
    others = [x for x in range(kp.shape[0]) if x != page]
    assert torch.equal(kk[others], want_k[others]) and torch.equal(vv[others], want_v[others])
    far = lens.clone()
    far[2] = table.shape[1] * 16 - 2              # tokens 2.. of this sequence are past the table
    status, out, kk, vv = run(lens=far)
    assert status == atlas.DEV_BAD_SEQLEN and torch.equal(out, good)
    far[2] = -3
    assert run(lens=far)[0] == atlas.DEV_BAD_SEQLEN
    for count in (-1, 7):
        n_new = torch.tensor([6, count, 6], dtype=torch.int32, device="cuda")
        status, out, kk, vv = run(n_new=n_new)
        assert status == atlas.DEV_BAD_SEQLEN and (out[1] == 99).all()
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(kk[page], clean_k[page])


@gpu
def test_captured_with_other_positions_at_replay():
    q, k, v, kp, vp, table, lens, pos = step("bf16", 2, 8, 2, 128, 16, 1, [30, 31], 3, 4)
    stream = torch.cuda.Stream()
    q_out = torch.empty_like(q)
    axis = atlas.rope_sections((16, 24, 24))
    with torch.cuda.stream(stream):
        atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos, pair_axis=axis, q_out=q_out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos, pair_axis=axis, q_out=q_out)
    torch.cuda.synchronize()
    pos.add_(123)
    lens.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    kp2, vp2 = kp.clone(), vp.clone()
    want = atlas.kv_append_rope(q, k, v, kp2, vp2, table, lens, pos, pair_axis=axis)
    assert torch.equal(q_out, want) and torch.equal(kp, kp2) and torch.equal(vp, vp2)


@gpu
def test_wrapper_refuses():
    q, k, v, kp, vp, table, lens, pos = step("bf16", 2, 4, 2, 128, 16, 3, [0, 1], 2, 6)
    ok = (q, k, v, kp, vp, table, lens, pos)

    def swap(i, x):
        return ok[:i] + (x,) + ok[i + 1:]

    for bad in (swap(0, q.float()), swap(0, q[:, :, :2]), swap(1, k.cpu()), swap(2, v[:, :1]),
                swap(3, kp[:, :1]), swap(5, table.long()), swap(5, table[:1]), swap(6, lens[:1]),
                swap(7, pos.long()), swap(7, pos[:, :1])):
        with pytest.raises(ValueError):
            atlas.kv_append_rope(*bad)
    for kw in (dict(pair_axis=(0, 1)), dict(inv_freq=[1.0]), dict(n_new=lens[:1]),
               dict(q_out=torch.empty_like(q[:, :1]))):
        with pytest.raises(ValueError):
            atlas.kv_append_rope(*ok, **kw)
    with pytest.raises(atlas.AtlasError):
        atlas.kv_append_rope(*ok, rot_dim=130)
    wide = torch.zeros((2, 4, 3, 256), dtype=torch.bfloat16, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        atlas.kv_append_rope(*swap(0, wide))
    with pytest.raises(ValueError):                    # one row for all: strides 0, 0, 0
        atlas.kv_append_rope(*swap(0, q[:1, :1, :1].expand(2, 4, 3, 128)))
    odd = torch.zeros(2 * 4 * 3 * 130, dtype=torch.bfloat16, device="cuda").view(2, 4, 3, 130)[..., :128]
    with pytest.raises(atlas.AtlasError):              # rows that do not start on 16 bytes
        atlas.kv_append_rope(*swap(0, odd))


@gpu
def test_broadcast_and_sliced_views_are_read_where_they_lie():
    q, k, v, kp, vp, table, lens, pos = step("bf16", 2, 4, 2, 128, 16, 3, [0, 1], 2, 7)
    heads = q[:, :1].expand(2, 4, 3, 128)              # one head's rows for all heads
    a = atlas.kv_append_rope(heads, k, v, kp, vp, table, lens, pos)
    assert torch.equal(a, atlas.kv_append_rope(heads.contiguous(), k, v, kp, vp, table, lens, pos))
    wide = torch.zeros((2, 4, 9, 136), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 3:6, :128] = q
    b = atlas.kv_append_rope(wide[:, :, 3:6, :128], k, v, kp, vp, table, lens, pos)
    assert torch.equal(b, atlas.kv_append_rope(q, k, v, kp, vp, table, lens, pos))
    one = k[:, :, 1:2]                                  # a single token out of several
    kp2, vp2 = kp.clone(), vp.clone()
    atlas.kv_append_rope(None, one, v[:, :, 1:2], kp, vp, table, lens, pos[:, :, 1:2].contiguous())
    atlas.kv_append_rope(None, one.contiguous(), v[:, :, 1:2].contiguous(), kp2, vp2, table, lens,
                         pos[:, :, 1:2].contiguous())
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
