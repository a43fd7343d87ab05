"""A cache under a budget: atlas_kv_weights, atlas_kv_select and atlas_kv_compact, each
against a plain form, and a run of them with the attention calls around them.

Tolerance of the weights.  A weight is 2^(s2 - lse2) summed over rows, with s2 the score
in log2 units.  Its relative error is ln 2 times the absolute error of s2 - lse2, plus
the exponential's 2^-22 and the sum's.  The score is a sum of D <= 128 products, exact in
bf16 inputs, rounded once each in fp32: at most D / 2 * 2^-24 * |q| |k| scale log2 e in
whatever order (the tensor core's truncating additions are at most twice a rounding, over
D / 8 steps), with |q| |k| scale <= 1.5^2 sqrt(D) for the rows drawn here (their norms
stay below 1.5 sqrt(D)): 64 * 2^-24 * 2.25 * 11.4 * 1.45 < 1.5e-4 worst case, and lse2
rounds by 2^-24 of itself (below 2^-19).  Rounding errors add up like their square root
rather than their number, so the tests hold the sums to 2e-5, a fifth of the worst case
and twice what the attention calls' fp32 outputs are held to."""
import ctypes
import functools
import math

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.operator_refs import key_weights, keys_to_keep, row_lse, widen
from tests.paging import page_kv

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
W_REL = 2e-5


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def fill(x, kw):
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def call_weights(lib, ptrs=(0x1000,) * 5, Hq=8, Hkv=2, D=128, P=16, scale=0.1, **kw):
    W = fill(atlas._Weights(), {**dict(batch=2, max_pages_per_seq=8, num_pages=16, q_len=4, dtype=1,
                                       weights=0x1000, row_tokens=128, accumulate=1), **kw})
    size = lib.atlas_kv_weights_workspace_size(Hq, Hkv, D, P, ctypes.byref(W))
    return lib.atlas_kv_weights(*ptrs, Hq, Hkv, D, P, scale, ctypes.byref(W)), size


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(q_len=0), 1), (dict(q_len=129), 1), (dict(num_pages=0), 1),
    (dict(row_tokens=0), 1), (dict(window=-1), 1), (dict(softcap=-1.0), 1),
    (dict(softcap=math.inf), 1), (dict(softcap=math.nan), 1), (dict(accumulate=2), 1),
    (dict(sm_count=-1), 1), (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(batch=65536), 1),
    (dict(D=96), 2), (dict(P=12), 2), (dict(P=4), 2), (dict(P=256), 2), (dict(dtype=2), 2)])
def test_weights_refusals(lib, kw, status):
    got, size = call_weights(lib, **kw)
    assert got == status and size == ctypes.c_size_t(-1).value


def test_weights_refuses_bad_pointers_and_scales(lib):
    for i in range(5):
        assert call_weights(lib, ptrs=tuple(None if k == i else 0x1000 for k in range(5)))[0] == 1
    assert call_weights(lib, ptrs=(0x1008,) + (0x1000,) * 4)[0] == 1
    assert call_weights(lib, weights=None)[0] == 1
    assert call_weights(lib, weights=0x1002)[0] == 1
    for scale in (math.nan, math.inf):
        assert call_weights(lib, scale=scale)[0] == 1
    assert lib.atlas_kv_weights(*(0x1000,) * 5, 8, 2, 128, 16, 0.1, None) == 1


def call_select(lib, w=0x1000, lens=0x1000, Hkv=2, **kw):
    S = fill(atlas._Select(), {**dict(batch=2, row_tokens=100, budget=10, keep_first=1, keep_recent=2,
                                      kept=0x1000, new_lens=0x1000), **kw})
    return lib.atlas_kv_select(w, lens, Hkv, ctypes.byref(S))


@pytest.mark.parametrize("kw", [dict(batch=0), dict(budget=0), dict(keep_first=-1),
                                dict(keep_recent=-1), dict(keep_first=9), dict(row_tokens=0),
                                dict(keep_first=2 ** 31 - 1, keep_recent=2 ** 31 - 1),
                                dict(kept=None), dict(new_lens=None), dict(w=None), dict(lens=None),
                                dict(Hkv=0), dict(w=0x1001), dict(kept_weights=0x1002),
                                dict(kept_weights=0x1000), dict(kept_weights=0x1000 + 4 * 2 * 2 * 100 - 4),
                                dict(kept_weights=0x1000 - 4 * 2 * 2 * 10 + 4),
                                dict(batch=70000), dict(budget=2 ** 31 - 1)])
def test_select_refusals(lib, kw):
    assert call_select(lib, **kw) == 1


def call_compact(lib, ptrs=(0x1000,) * 5, Hkv=2, D=128, P=16, **kw):
    C = fill(atlas._Compact(), {**dict(batch=2, max_pages_per_seq=4, num_pages=8, max_kept=10,
                                       kv_dtype=1), **kw})
    return lib.atlas_kv_compact(*ptrs, Hkv, D, P, ctypes.byref(C))


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(max_pages_per_seq=0), 1), (dict(num_pages=0), 1), (dict(max_kept=0), 1),
    (dict(new_page_table=0x1000), 1), (dict(Hkv=0), 1), (dict(Hkv=4096), 1), (dict(D=80), 2),
    (dict(P=12), 2), (dict(kv_dtype=3), 2), (dict(ptrs=(0x1008,) + (0x1000,) * 4), 1),
    (dict(ptrs=(None,) + (0x1000,) * 4), 1),
    (dict(ptrs=(0x1000,) * 5), 1), (dict(ptrs=(0x10000, 0x10000 + 8 * 2 * 16 * 256 - 16) + (0x1000,) * 3), 1),
    (dict(ptrs=(0x1000,) * 3 + (None, 0x1000)), 1)])
def test_compact_refusals(lib, kw, status):
    assert call_compact(lib, **kw) == status


def test_plain_forms_on_cases_worked_by_hand():
    assert keys_to_keep([5, 1, 9, 9, 2, 0], 6, 4, 1, 1) == [0, 2, 3, 5]
    assert keys_to_keep([1, 7, 7, 7, 7], 5, 2, 0, 0) == [1, 2]            # ties: lower index
    assert keys_to_keep([math.nan, 0.0, -0.0, 1], 4, 2, 0, 0) == [1, 3]
    assert keys_to_keep([3, 2], 2, 4, 1, 1) == [0, 1]
    # two keys with scores 0 and ln 3: weights 1/4 and 3/4
    k = np.array([0.0, math.log(3)]).reshape(1, 1, 2, 1)
    q = np.ones((1, 2, 1, 1))
    lse = row_lse(q, k, [2], 1.0)
    assert np.allclose(lse, math.log(4))
    assert np.allclose(key_weights(q, k, [2], lse, 1.0), [[[0.5, 1.5]]])


# ------------------------------------------------------------------ weights
def problem(dtype, Hq, Hkv, D, P, q_len, lens, seed):
    r = np.random.default_rng(seed)

    def draw(*shape):
        return torch.from_numpy(r.standard_normal(shape, dtype=np.float32)).to(DT[dtype])

    q, k = draw(len(lens), Hq, q_len, D), draw(len(lens), Hkv, max(lens), D)
    kp, _, table = page_kv(k.float().numpy(), k.float().numpy(), lens, P, seed=seed, pad_page=-7)
    return q, k, (q.cuda(), torch.from_numpy(kp).to(DT[dtype]).cuda(), torch.from_numpy(table).cuda(),
                  torch.tensor(lens, dtype=torch.int32, device="cuda"))


WEIGHTS = [
    # dtype, Hq, Hkv, D, P, q_len, lens, options
    ("bf16", 8, 2, 128, 16, 1, [300, 1, 129], {}),
    ("bf16", 4, 4, 64, 64, 1, [64, 65, 4000], {}),
    ("f32", 8, 1, 64, 16, 1, [127, 1000], {}),
    ("f32", 4, 2, 128, 8, 3, [3, 500], dict(softcap=5.0)),
    ("bf16", 16, 2, 128, 32, 5, [5, 200, 1500], dict(window=70)),
    ("bf16", 8, 1, 64, 128, 32, [32, 900], dict(ragged=[32, 7])),
    ("bf16", 8, 2, 128, 16, 40, [100, 1000, 41], dict(ragged=[40, 1, 0])),
    ("bf16", 6, 2, 128, 64, 90, [600, 90], dict(softcap=2.0)),
    ("bf16", 4, 1, 128, 16, 257, [257, 1200], {}),
    ("bf16", 8, 2, 64, 16, 128, [128, 777], dict(window=100)),
    ("bf16", 2, 1, 128, 32, 600, [600, 601], dict(ragged=[600, 333])),
    ("bf16", 2, 2, 64, 8, 300, [1100], dict(scale=-0.2)),
    ("bf16", 8, 1, 128, 16, 25, [3000, 25, 150], dict(window=2 ** 31 - 1)),
    ("bf16", 4, 1, 64, 32, 129, [129, 2500], dict(window=2 ** 31 - 1, ragged=[0, 128])),
    ("bf16", 8, 2, 128, 128, 16, [1029, 17], dict(window=1)),
    ("f32", 6, 2, 64, 32, 100, [100, 333], dict(ragged=[100, 50])),
    ("f32", 2, 2, 64, 32, 3, [100, 333], dict(window=2 ** 31 - 1, ragged=[0, 2])),
    ("f32", 4, 2, 128, 16, 65, [400], dict(window=33, softcap=4.0)),
    ("f32", 4, 1, 128, 64, 200, [200, 1000, 333], dict(ragged=[200, 3, 0])),
    ("f32", 2, 1, 64, 16, 300, [700, 300, 511], {}),
    ("f32", 8, 2, 128, 8, 40, [900, 41], dict(window=100)),
    ("f32", 2, 1, 128, 128, 257, [257, 513], dict(scale=-0.06)),
    ("f32", 3, 1, 64, 8, 5, [5, 300], {}),
    ("f32", 2, 1, 128, 8, 1, [1, 700], dict(window=300)),
    ("f32", 2, 2, 64, 64, 2, [2, 129], dict(ragged=[0, 1])),
    ("f32", 8, 2, 64, 128, 16, [2100, 16, 129], {}),
    ("f32", 4, 1, 128, 16, 16, [5000, 17], dict(ragged=[16, 0], softcap=3.0)),
    # more than 64 columns of fp32: planned for few SMs, K goes past them in several launches
    ("f32", 4, 1, 128, 64, 60, [60, 1000, 333], dict(ragged=[60, 3, 0], sm_count=1)),
    ("f32", 6, 2, 64, 8, 40, [900, 41], dict(window=100, sm_count=1)),
    ("f32", 4, 2, 128, 16, 33, [400], dict(window=33, softcap=4.0, sm_count=2)),
    ("f32", 2, 1, 64, 16, 128, [700, 128, 511], dict(ragged=[128, 33, 128], sm_count=1)),
]


@gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,D,P,q_len,lens,opt", WEIGHTS)
def test_weights_match_the_plain_form(dtype, Hq, Hkv, D, P, q_len, lens, opt):
    q, k, dev = problem(dtype, Hq, Hkv, D, P, q_len, lens, 40 + q_len)
    scale, ragged = opt.get("scale", D ** -0.5), opt.get("ragged")
    var = dict(window=opt.get("window", 0), softcap=opt.get("softcap", 0.0))
    lse = row_lse(widen(q), widen(k), lens, scale, ragged, **var)
    lse = np.float32(lse)                                    # the input: these values exactly
    want = key_weights(widen(q), widen(k), lens, lse.astype(np.float64), scale, ragged, **var)
    if ragged:
        for b, n in enumerate(ragged):                       # padding rows: NaN, never used
            dev[0][b, :, n:] = float("nan")
    T = dev[2].shape[1] * P + 5                              # rows longer than the table
    rng = np.random.default_rng(1)
    start = torch.from_numpy(rng.random((len(lens), Hkv, T), dtype=np.float32)).cuda()
    kw = dict(q_lens=None if ragged is None else torch.tensor(ragged, dtype=torch.int32, device="cuda"),
              sm_count=opt.get("sm_count", 0), **var)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (*dev, torch.from_numpy(lse).cuda(), Hq, Hkv, D, P, scale)
    fresh = atlas.kv_weights(*args, weights=start.clone(), accumulate=False, status=status, **kw)
    added = atlas.kv_weights(*args, weights=start.clone(), status=status, **kw)
    assert int(status.item()) == 0
    for b, L in enumerate(lens):
        got = widen(fresh[b, :, :L])
        assert np.isfinite(got).all()
        assert (np.abs(got - want[b, :, :L]) <= W_REL * want[b, :, :L] + 1e-30).all()
        both = widen(start[b, :, :L]) + want[b, :, :L]
        assert (np.abs(widen(added[b, :, :L]) - both) <= (W_REL + 2.0 ** -23) * both).all()
        for x in (fresh, added):                             # nothing behind the end is touched
            assert torch.equal(x[b, :, L:], start[b, :, L:])
    again = atlas.kv_weights(*args, weights=start.clone(), accumulate=False, **kw)
    assert torch.equal(again, fresh)                         # the same bits each time


@gpu
@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("bf16", 70), ("bf16", 300), ("f32", 1), ("f32", 12), ("f32", 70)])
def test_weights_of_the_attention_calls_lse_sum_to_the_rows(dtype, q_len):
    """Each row's weights sum to 1, so a (sequence, kv head) collects one per row."""
    q, k, dev = problem(dtype, 8, 2, 128, 16, q_len, [q_len + 400, q_len + 3], 9)
    lse = torch.empty(q.shape[:3], device="cuda")
    atlas.suffix(dev[0], dev[1], dev[1], dev[2], dev[3], 8, 2, 128, 16, 0.09, lse=lse)
    w = atlas.kv_weights(*dev, lse, 8, 2, 128, 16, 0.09)
    total = widen(w).sum(-1)
    # lse is good to 1e-4 (2e-5 in fp32): that much of each row's 1
    assert np.abs(total / (4 * q_len) - 1).max() <= (1.5e-4 if dtype == "bf16" else 5e-5)


@gpu
@pytest.mark.parametrize("dtype,q_len,sms", [("bf16", 2, 0), ("bf16", 300, 0), ("f32", 1, 0), ("f32", 2, 0),
                                             ("f32", 100, 0), ("f32", 100, 1)])
def test_weights_of_rows_that_saw_nothing_and_of_bad_sequences(dtype, q_len, sms):
    lens = [q_len + 50, q_len + 700, q_len + 10]
    q, k, dev = problem(dtype, 4, 2, 64, 16, q_len, lens, 3)
    lse = torch.from_numpy(np.float32(row_lse(widen(q), widen(k), lens, 0.125))).cuda()
    args = (4, 2, 64, 16, 0.125)
    kv_weights = functools.partial(atlas.kv_weights, sm_count=sms)
    good = kv_weights(*dev, lse, *args)
    # one head of the first sequence saw nothing: it adds nothing
    none = lse.clone()
    none[0, 1] = -math.inf
    rest = lse.clone()
    rest[0, 1] = 1e30                                        # exp(s - 1e30) = 0
    a, b = kv_weights(*dev, none, *args), kv_weights(*dev, rest, *args)
    assert torch.equal(a, b) and not torch.equal(a[0], good[0]) and torch.equal(a[1:], good[1:])
    for bad in (q_len - 1, -1, good.shape[2] + 1):
        bad_lens = dev[3].clone()
        bad_lens[1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = kv_weights(*dev[:3], bad_lens, lse, *args, status=status, accumulate=False,
                       weights=torch.full_like(good, 7.0))
        assert int(status.item()) == atlas.DEV_BAD_SEQLEN and (w[1] == 7).all()
        assert torch.equal(w[0, :, :lens[0]], good[0, :, :lens[0]])
        assert torch.equal(w[2, :, :lens[2]], good[2, :, :lens[2]])
    for bad in (-1, 3):
        counts = torch.tensor([q_len, bad if bad < 0 else q_len + 1, q_len], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv_weights(*dev, lse, *args, status=status, q_lens=counts)
        assert int(status.item()) == atlas.DEV_BAD_SEQLEN
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    short = torch.zeros((3, 2, lens[1] - 1), device="cuda")  # the weights' rows are too short for it
    kv_weights(*dev, lse, *args, status=status, weights=short)
    assert int(status.item()) == atlas.DEV_BAD_SEQLEN and (short[1] == 0).all()
    table = dev[2].clone()
    table[1, 0] = dev[1].shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = kv_weights(dev[0], dev[1], table, dev[3], lse, *args, status=status, accumulate=False,
                   weights=torch.full_like(good, 7.0))
    assert int(status.item()) == atlas.DEV_BAD_PAGE and (w[1, :, :16] == 7).all()
    assert torch.equal(w[1, :, 512:lens[1]], good[1, :, 512:lens[1]])
    assert torch.equal(w[0, :, :lens[0]], good[0, :, :lens[0]])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,G,D,P,q_len,L", [(3, 8, 4, 128, 64, 64, 5000), (3, 8, 4, 64, 64, 64, 5000),
                                                 (6, 4, 8, 128, 32, 9, 9000), (4, 8, 4, 64, 16, 1, 9000)])
def test_weights_are_the_same_each_time_whatever_the_caches_hold(dtype, B, Hkv, G, D, P, q_len, L):
    """Many CTAs streaming a long context, from a cold L2 and from a warm one: copies land
    late or early, the bits stay, and they are the plain form's within its tolerance."""
    g = torch.Generator(device="cuda").manual_seed(L + D)
    pages = -(-L // P)
    k = torch.randn((B * pages, Hkv, P, D), generator=g, device="cuda").to(DT[dtype])
    q = torch.randn((B, Hkv * G, q_len, D), generator=g, device="cuda").to(DT[dtype])
    table = torch.randperm(B * pages, generator=g, device="cuda").int().reshape(B, pages)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    rows = k[table.long()].transpose(1, 2).reshape(B, Hkv, pages * P, D)[:, :, :L].double()
    s = (q.double().reshape(B, Hkv, G * q_len, D) @ rows.transpose(2, 3) * D ** -0.5).reshape(B, Hkv, G, q_len, L)
    pos = torch.arange(L - q_len, L, device="cuda")[:, None]
    s = s.masked_fill(torch.arange(L, device="cuda")[None] > pos, -math.inf)
    lse = torch.logsumexp(s, -1).float()
    want = torch.exp(s - lse.double()[..., None]).sum((2, 3))
    cold = torch.empty(100_000_000, device="cuda")           # 400 MB: more than the L2
    first = None
    for n in range(12):
        if n % 2 == 0:
            cold.fill_(n)
        w = atlas.kv_weights(q, k, table, lens, lse.reshape(B, Hkv * G, q_len), Hkv * G, Hkv, D, P, D ** -0.5)
        first = w if first is None else first
        assert torch.equal(w, first)
    assert ((first[:, :, :L].double() - want).abs() <= W_REL * want + 1e-30).all()


# ------------------------------------------------------------------ selection
def totals(kind, B, Hkv, T, seed):
    r = np.random.default_rng(seed)
    w = r.standard_exponential((B, Hkv, T)).astype(np.float32) ** 4
    if kind == "ties":
        w = np.float32(r.integers(0, 3, (B, Hkv, T)))
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":                     # every kind of value, -0 and 0, NaN, infinities
        pick = np.float32([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, -1e-45, 3e38, 1.0, -1.0])
        w = pick[r.integers(0, len(pick), (B, Hkv, T))]
    return w


SELECT = [
    # kind, B, Hkv, T, lens, budget, first, recent
    ("plain", 3, 2, 700, [700, 129, 512], 128, 4, 16),
    ("plain", 2, 3, 5000, [5000, 4999], 1000, 0, 0),
    ("plain", 2, 1, 40000, [39999, 17], 777, 16, 100),
    ("ties", 2, 2, 9000, [9000, 8191], 4096, 1, 1),
    ("equal", 1, 2, 3000, [2999], 1500, 10, 20),
    ("odd", 3, 2, 1000, [1000, 999, 501], 500, 2, 3),
    ("odd", 1, 1, 20000, [20000], 19999, 0, 1),
    ("plain", 4, 1, 64, [0, 1, 64, 33], 32, 16, 16),        # nothing is left to choose
    ("plain", 2, 1, 64, [64, 5], 1, 0, 0),
    ("plain", 2, 1, 64, [64, 5], 1, 1, 0),
    ("plain", 1, 2, 300, [300], 1000, 0, 0),                # a budget beyond the row
    ("ties", 1, 1, 420000, [419999], 5000, 4, 64),          # too long to stay in shared memory
    ("plain", 20, 17, 700, [700, 333, 0, 5] * 5, 300, 2, 9),  # more rows than two for each SM
    ("ties", 39, 8, 300, [300, 299, 13] * 13, 100, 0, 0),
    ("odd", 1, 2, 4096, [4096], 1000, 3, 0),
    ("plain", 1, 2, 4097, [4097], 1000, 3, 0),
]


@gpu
@pytest.mark.parametrize("kind,B,Hkv,T,lens,budget,first,recent", SELECT)
def test_select_matches_the_plain_form(kind, B, Hkv, T, lens, budget, first, recent):
    w = totals(kind, B, Hkv, T, T + budget)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new, kept_w = atlas.kv_select(torch.from_numpy(w).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        budget, keep_first=first, keep_recent=recent, status=status)
    assert int(status.item()) == 0
    assert new.tolist() == [min(x, budget) for x in lens]
    kept, kept_w = kept.cpu().numpy(), kept_w.cpu().numpy()
    for b in range(B):
        for g in range(Hkv):
            want = keys_to_keep(w[b, g].tolist(), lens[b], budget, first, recent)
            assert kept[b, g].tolist() == want + [-1] * (budget - len(want))
            assert np.array_equal(kept_w[b, g, :len(want)], w[b, g, want], equal_nan=True)
            assert (kept_w[b, g, len(want):] == 0).all()


@gpu
def test_select_counts_a_bad_length_as_none():
    w = torch.rand((3, 2, 50), device="cuda")
    lens = torch.tensor([50, 51, -1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new, kept_w = atlas.kv_select(w, lens, 10, status=status)
    assert int(status.item()) == atlas.DEV_BAD_SEQLEN and new.tolist() == [10, 0, 0]
    assert (kept[1:] == -1).all() and (kept_w[1:] == 0).all() and (kept[0] >= 0).all()


# ------------------------------------------------------------------ compaction
def pools(dtype, B, Hkv, D, P, width, fresh, seed):
    r = np.random.default_rng(seed)
    num = B * (width + fresh) + 2
    ids = r.permutation(num).astype(np.int32)
    kp, vp = (torch.from_numpy(r.standard_normal((num, Hkv, P, D), dtype=np.float32)).to(DT[dtype]).cuda()
              for _ in range(2))
    table = torch.from_numpy(ids[:B * width].reshape(B, width)).cuda()
    new = torch.from_numpy(ids[B * width:B * (width + fresh)].reshape(B, fresh)).cuda() if fresh else None
    return kp, vp, table, new


def moved(pool, table, to, kept, lens):
    out = pool.clone()
    P = pool.shape[2]
    table, to, kept = table.cpu(), to.cpu(), kept.cpu()
    for b, n in enumerate(lens):
        for g in range(pool.shape[1]):
            j, t = torch.arange(n), kept[b, g, :n].long()
            src, dst = table[b, t // P].long(), to[b, j // P].long()
            out[dst.cuda(), g, (j % P).cuda()] = pool[src.cuda(), g, (t % P).cuda()]
    return out


@gpu
@pytest.mark.parametrize("dtype,Hkv,D,P,lens,L", [
    ("bf16", 2, 128, 16, [100, 33, 0], 240), ("bf16", 1, 64, 64, [129, 1, 64], 192),
    ("f32", 2, 64, 8, [77, 80, 5], 80), ("f32", 1, 128, 128, [300, 2, 301], 640),
    ("bf16", 1, 128, 8, [1500, 1499, 700], 2048),
    ("bf16", 1, 64, 8, [900, 40, 0], 65600),                # a table of 8200 pages
    ("bf16", 2, 64, 32, [20000, 8193, 4096], 24000)])       # several batches of indices
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_moves_the_kept_rows(dtype, Hkv, D, P, lens, L, in_place):
    n = max(lens)
    kp, vp, table, new = pools(dtype, 3, Hkv, D, P, L // P, 0 if in_place else -(-n // P), L)
    r = np.random.default_rng(2)
    kept = np.full((3, Hkv, n + 3), -1, np.int32)
    for b in range(3):
        for g in range(Hkv):
            kept[b, g, :lens[b]] = np.sort(r.choice(L, lens[b], replace=False))
    if not in_place and lens[0] > 50:                         # any order, repeats too
        kept[0, 0, :lens[0]] = r.integers(0, L, lens[0])
    if in_place:                                              # a long prefix that stays where it is
        kept[1, 0, :lens[1]] = np.arange(lens[1])
    kept = torch.from_numpy(kept).cuda()
    want = [moved(x, table, table if in_place else new, kept, lens) for x in (kp, vp)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    atlas.kv_compact(kp, vp, table, kept, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     new_page_table=new, status=status)
    assert int(status.item()) == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


@gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_reports_and_skips(in_place):
    kp, vp, table, new = pools("bf16", 2, 1, 64, 16, 6, 0 if in_place else 2, 5)
    kept = torch.arange(0, 64, 2, dtype=torch.int32, device="cuda").expand(2, 1, 32).contiguous()
    lens = torch.tensor([32, 20], dtype=torch.int32, device="cuda")
    to = table if in_place else new
    clean = kp.clone(), vp.clone()

    def run(table=table, kept=kept, lens=lens, new=new):
        kk, vv = clean[0].clone(), clean[1].clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        atlas.kv_compact(kk, vv, table, kept, lens, new_page_table=new, status=status)
        return int(status.item()), kk, vv

    whole = run()
    assert whole[0] == 0
    for n in (-1, 33):                                        # sequence 1 does not fit
        status, kk, vv = run(lens=torch.tensor([32, n], dtype=torch.int32, device="cuda"))
        assert status == atlas.DEV_BAD_SEQLEN
        assert torch.equal(kk, moved(clean[0], table, to, kept, [32, 0]))
    odd = kept.clone()
    odd[1, 0, 3] = 96                                         # past the table
    odd[1, 0, 5] = -1
    if in_place:
        odd[1, 0, 9] = 8                                      # below its own place
    status, kk, vv = run(kept=odd)
    assert status == atlas.DEV_BAD_SEQLEN
    for j in (3, 5) + ((9,) if in_place else ()):             # these rows stay, the others move
        at = (int(to[1, j // 16]), 0, j % 16)
        assert torch.equal(kk[at], clean[0][at]) and torch.equal(vv[at], clean[1][at])
        kk[at], vv[at] = whole[1][at], whole[2][at]
    assert torch.equal(kk, whole[1]) and torch.equal(vv, whole[2])
    broken = table.clone()
    broken[0, 3] = -4                                         # sources of rows 24..31
    status, kk, vv = run(table=broken)
    assert status == atlas.DEV_BAD_PAGE
    for j in range(24, 32):
        at = (int(to[0, j // 16]), 0, j % 16)
        assert torch.equal(kk[at], clean[0][at])
        kk[at], vv[at] = whole[1][at], whole[2][at]
    assert torch.equal(kk, whole[1]) and torch.equal(vv, whole[2])


# ------------------------------------------------------------------ streams, graphs, refusals
def cut(w, k, v, table, lens, budget, **out):
    kept, new, kept_w = atlas.kv_select(w, lens, budget, keep_first=2, keep_recent=9, **out)
    atlas.kv_compact(k, v, table, kept, new)
    return kept, new, kept_w


@gpu
@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("bf16", 40), ("bf16", 200), ("f32", 1), ("f32", 16),
                                         ("f32", 200)])
def test_captured_and_replayed_with_other_lengths(dtype, q_len):
    q, k, dev = problem(dtype, 8, 2, 128, 16, q_len, [900, 700], 21)
    v_pages = torch.randn_like(dev[1])
    lse = torch.from_numpy(np.float32(row_lse(widen(q), widen(k), [900, 700], 0.09))).cuda()
    shape = (2, 2, dev[2].shape[1] * 16)
    pools0 = dev[1].clone(), v_pages.clone()
    outs = dict(kept=torch.empty((2, 2, 300), dtype=torch.int32, device="cuda"),
                new_lens=torch.empty(2, dtype=torch.int32, device="cuda"),
                kept_weights=torch.empty((2, 2, 300), device="cuda"))
    w = torch.zeros(shape, device="cuda")
    stream = torch.cuda.Stream()

    def run():
        atlas.kv_weights(*dev, lse, 8, 2, 128, 16, 0.09, weights=w, accumulate=False)
        cut(w, dev[1], v_pages, dev[2], dev[3], 300, **outs)

    with torch.cuda.stream(stream):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run()
    for lens in ([900, 700], [300, q_len], [640, 333]):
        torch.cuda.synchronize()
        lens = torch.tensor([max(x, q_len) for x in lens], dtype=torch.int32)
        dev[3].copy_(lens)
        dev[1].copy_(pools0[0])
        v_pages.copy_(pools0[1])
        w.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kk, vv = pools0[0].clone(), pools0[1].clone()
        ww = atlas.kv_weights(dev[0], kk, *dev[2:], lse, 8, 2, 128, 16, 0.09, accumulate=False,
                              weights=torch.full(shape, 5.0, device="cuda"))
        kept, new, kept_w = cut(ww, kk, vv, dev[2], dev[3], 300)
        assert torch.equal(w, ww) and torch.equal(outs["kept"], kept) and torch.equal(outs["new_lens"], new)
        assert torch.equal(outs["kept_weights"], kept_w)
        assert torch.equal(dev[1].isnan(), kk.isnan()) and torch.equal(dev[1].nan_to_num(), kk.nan_to_num())
        assert torch.equal(v_pages, vv)


@gpu
def test_two_streams_at_once():
    """Calls on two streams with tensors of their own give what they give alone."""
    sides = []
    for seed in (31, 32):
        q, k, dev = problem("bf16", 8, 1, 64, 32, 150, [3000, 150, 1111], seed)
        lse = torch.from_numpy(np.float32(row_lse(widen(q), widen(k), [3000, 150, 1111], 0.125))).cuda()
        alone = atlas.kv_weights(*dev, lse, 8, 1, 64, 32, 0.125)
        kk, vv = dev[1].nan_to_num(), torch.randn_like(dev[1])
        pools = kk.clone(), vv.clone()
        sides.append((dev, lse, alone, kk, vv, pools, cut(alone, kk, vv, dev[2], dev[3], 700)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    got = [None, None]
    for _ in range(5):
        for i, (dev, lse, alone, kk, vv, pools, want) in enumerate(sides):
            with torch.cuda.stream(streams[i]):
                w = atlas.kv_weights(*dev, lse, 8, 1, 64, 32, 0.125)
                a, b = pools[0].clone(), pools[1].clone()
                got[i] = w, a, b, cut(w, a, b, dev[2], dev[3], 700)
    torch.cuda.synchronize()
    for (dev, lse, alone, kk, vv, pools, want), (w, a, b, out) in zip(sides, got):
        assert torch.equal(w, alone) and torch.equal(a, kk) and torch.equal(b, vv)
        assert all(torch.equal(x, y) for x, y in zip(out, want))


@gpu
def test_wrappers_refuse():
    q, k, dev = problem("bf16", 4, 2, 64, 16, 3, [40, 30], 1)
    lse = torch.zeros(q.shape[:3], device="cuda")
    ok = (*dev, lse)

    def swap(i, x):
        return ok[:i] + (x,) + ok[i + 1:]

    for bad in (swap(0, dev[0].float()), swap(0, dev[0][:, :, :2]), swap(1, dev[1].cpu()), swap(2, dev[2][:1]),
                swap(2, dev[2].long()), swap(3, dev[3][:1]), swap(4, lse.double()), swap(4, lse[:, :2].contiguous())):
        with pytest.raises(ValueError):
            atlas.kv_weights(*bad, 4, 2, 64, 16, 0.1)
    for kw in (dict(weights=torch.zeros((2, 1, 64), device="cuda")), dict(q_lens=dev[3][:1]),
               dict(weights=torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)),
               dict(weights=torch.zeros((2, 2, 128), device="cuda")[:, :, ::2])):
        with pytest.raises(ValueError):
            atlas.kv_weights(*ok, 4, 2, 64, 16, 0.1, **kw)
    with pytest.raises(ValueError):
        atlas.kv_weights(*ok, 8, 2, 64, 16, 0.1)               # q has 4 heads
    w = torch.rand((2, 2, 64), device="cuda")
    for args in ((w[0], dev[3], 8), (w, dev[3][:1], 8), (w.double(), dev[3], 8)):
        with pytest.raises(ValueError):
            atlas.kv_select(*args)
    for kw in (dict(keep_first=5, keep_recent=4), dict(keep_first=-1)):
        with pytest.raises(atlas.AtlasError):
            atlas.kv_select(w, dev[3], 8, **kw)
    with pytest.raises(atlas.AtlasError):
        atlas.kv_select(w, dev[3], 0)
    kept, new, _ = atlas.kv_select(w, dev[3], 8)
    for args in ((dev[1], dev[1][:1], dev[2], kept, new), (dev[1], dev[1], dev[2], kept[:1], new),
                 (dev[1], dev[1], dev[2], kept.long(), new), (dev[1], dev[1], dev[2], kept, new[:1])):
        with pytest.raises(ValueError):
            atlas.kv_compact(*args)
    with pytest.raises(ValueError):
        atlas.kv_compact(dev[1], dev[1].clone(), dev[2], kept, new, new_page_table=dev[2][:1])


@gpu
def test_a_workspace_too_small_is_refused():
    q, k, dev = problem("bf16", 8, 1, 64, 16, 300, [1000], 2)
    lse = torch.zeros(q.shape[:3], device="cuda")
    with pytest.raises(atlas.AtlasError):
        atlas.kv_weights(*dev, lse, 8, 1, 64, 16, 0.1,
                         workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@gpu
def test_far_offsets_in_a_large_pool():
    """Pages behind 2^31 elements of the pool, for every operator that addresses it."""
    P, Hkv, D, last = 128, 8, 128, 17000                 # 17000 pages: 2.2e9 bf16 elements
    kp = torch.zeros((last + 1, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    small = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    far = torch.tensor([[last, last - 1, last - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn((1, h, 300, D), generator=g, device="cuda").to(torch.bfloat16) for h in (8, 8, 16))
    pos = torch.arange(300, dtype=torch.int32, device="cuda")[None]
    zero, full = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, 300))
    got = []
    for table in (small, far):
        qr = atlas.kv_append_rope(q, k, v, kp, vp, table, zero, pos)
        lse = torch.empty((1, 16, 300), device="cuda")
        out = atlas.prefill(qr, kp, vp, table, full, 16, 8, D, P, 0.09, lse=lse)
        crossed = atlas.cross(qr, kp, vp, table, full, 16, 8, D, P, 0.09)
        w = atlas.kv_weights(qr, kp, table, full, lse, 16, 8, D, P, 0.09)
        one = atlas.kv_weights(qr[:, :, -1:].contiguous(), kp, table, full, lse[:, :, -1:].contiguous(), 16, 8, D, P, 0.09)
        kept, new, _ = atlas.kv_select(w, full, 200)
        atlas.kv_compact(kp, vp, table, kept, new)
        got.append((qr, out, crossed, w, one, kept, kp[table[0].long()], vp[table[0].long()]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    del kp, vp, got
    torch.cuda.empty_cache()
