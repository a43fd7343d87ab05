"""Attention of sequences that share prefixes (atlas_attn_shared) against a plain fp64 form:
groups of all sizes, prefixes and own caches from one key on, ragged rows, every kernel path.

Tolerances are those of the causal calls (gpu_helpers), since the arithmetic is theirs: fp32
1e-5 of the largest |out|, bf16 inputs with fp32 output 2e-3, a bf16 output the rounding of the
fp32 one.  lse: fp32 2e-5, bf16 1e-4, as there."""
import ctypes

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.gpu_helpers import BF16_ABS, F32_REL
from tests.operator_refs import widen
from tests.paging import page_kv
from tests.serving_refs import shared_rows

SIZE_MAX = ctypes.c_size_t(-1).value
gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    _build.build()
    return atlas.load_library()


def launch(**kw):
    L = atlas._Launch()
    L.batch, L.max_pages_per_seq, L.num_pages, L.q_len = 4, 8, 64, 1
    L.q_dtype = L.kv_dtype = L.out_dtype = 1
    L.out = 0x1000
    for k, v in kw.items():
        setattr(L, k, v)
    return L


def prefixes(**kw):
    S = atlas._Shared(0x1000, 0x1000, 0x1000, 2, 16)
    for k, v in kw.items():
        setattr(S, k, v)
    return S


def ws(lib, S=None, Hq=8, Hkv=2, D=128, P=16, **kw):
    return lib.atlas_attn_shared_workspace_size(Hq, Hkv, D, P, ctypes.byref(S or prefixes()),
                                                ctypes.byref(launch(**kw)))


def call(lib, S, L, ptrs=(0x1000,) * 5, scale=0.1):
    return lib.atlas_attn_shared(*ptrs, 8, 2, 128, 16, ctypes.c_float(scale),
                                 ctypes.byref(S) if S else None, ctypes.byref(L) if L else None)


@pytest.mark.parametrize("S,kw", [
    (None, dict(window=4)), (None, dict(window=-1)), (None, dict(phase=1)), (None, dict(phase=2)),
    (None, dict(chunk_range=0x1000)), (None, dict(Hq=7)), (None, dict(D=96)), (None, dict(P=12)),
    (None, dict(q_len=0)), (None, dict(batch=0)), (None, dict(q_len=129)), (None, dict(sm_count=-1)),
    (None, dict(split_tokens=32)), (None, dict(q_dtype=0)), (None, dict(out_dtype=2)),
    (dict(n_groups=0), {}), (dict(n_groups=5), {}), (dict(n_groups=-1), {}),
    (dict(max_prefix_pages=0), {}), (dict(max_prefix_pages=-1), {}),
    (dict(max_prefix_pages=1 << 30), {})])
def test_refusals(lib, S, kw):
    assert ws(lib, **kw, S=prefixes(**(S or {}))) == SIZE_MAX


def test_workspace_holds_the_states_of_both_parts(lib):
    # rows of 128 floats and (m, l): own 128 keys and a prefix of 256 in splits of 64
    rows, own, pre = 4 * 8, 2, 4
    n = ws(lib, split_tokens=64)
    acc = rows * 128 * 4
    own_bytes = (own * acc + rows * own * 8 + 255) // 256 * 256
    assert n == own_bytes + pre * acc + rows * pre * 8
    assert ws(lib) != SIZE_MAX and ws(lib, batch=4, S=prefixes(n_groups=4)) != SIZE_MAX
    assert atlas.shared_workspace_size((4, 8, 1, 128), 8, 2, 128, 16, 8, 2, 16, 64, split_tokens=64) == n
    with pytest.raises(atlas.AtlasError):
        atlas.shared_workspace_size((4, 8, 1, 128), 8, 2, 128, 16, 8, 5, 16, 64)
    # more SMs than any device has change nothing more
    assert ws(lib, sm_count=2 ** 31 - 1) == ws(lib, sm_count=1 << 20) != SIZE_MAX


@pytest.mark.parametrize("B,groups,q_len,prefix_pages,whole", [
    (1, 1, 20, 1000, False), (1, 1, 20, 100, True), (2, 2, 20, 1000, True), (8, 8, 20, 1000, True), (8, 8, 5, 1000, True), (64, 64, 75, 125, True),
    (32, 4, 20, 1000, False), (64, 1, 5, 1000, False), (64, 1, 64, 1000, True)])
def test_tiles_of_their_own_where_a_gather_fills_no_more(lib, B, groups, q_len, prefix_pages, whole):
    """Rows of a sequence alone in its group, or that fill tiles, are not gathered (as the sizes tell), where
    8 kv heads leave a tile to 16 of 152 SMs at most, or it has 33 blocks at most."""
    def size(flags):
        return ws(lib, prefixes(n_groups=groups, max_prefix_pages=prefix_pages), Hq=32, Hkv=8, batch=B, q_len=q_len,
                  max_pages_per_seq=100, debug_flags=flags, sm_count=152)
    own, gathered = size(atlas.DEBUG_SHARED_WHOLE), size(atlas.DEBUG_SHARED_TC)
    assert own != gathered and size(0) == (own if whole else gathered)


def serving(lib, B, q_len, own, prefix, heads=(32, 8), groups=1, dtype=1, P=16, **kw):
    """Workspace of B sequences of q_len rows, tables of that many own and prefix keys."""
    return ws(lib, prefixes(n_groups=groups, max_prefix_pages=-(-prefix // P)), Hq=heads[0], Hkv=heads[1], P=P,
              batch=B, q_len=q_len, max_pages_per_seq=-(-own // P), q_dtype=dtype, kv_dtype=dtype, out_dtype=dtype, **kw)


@pytest.mark.parametrize("B,q_len,own,prefix,heads", [
    (255, 1024, 1024, 1000, (32, 8)), (256, 1024, 1024, 1000, (32, 8)), (300, 1024, 1024, 1000, (32, 8)),
    (2048, 128, 1024, 1000, (32, 8)), (2049, 128, 1024, 1000, (32, 8)), (128, 1024, 4096, 1000, (64, 8))])
def test_batches_of_more_tiles_than_a_grid_of_splits_has(lib, B, q_len, own, prefix, heads):
    """65535 tiles of own keys and more, whose rows have tiles over all their keys."""
    assert serving(lib, B, q_len, own, prefix, heads) != SIZE_MAX


@pytest.mark.parametrize("B,q_len,own,prefix,dtype", [
    (64, 300, 2048, 32768, 1), (64, 300, 2048, 32768, 0), (512, 300, 32768, 32768, 1), (512, 300, 32768, 32768, 0),
    (512, 320, 32768, 32768, 1), (256, 256, 131072, 131072, 1), (256, 256, 131072, 131072, 0),
    (4, 8192, 131072, 131072, 1), (4, 8192, 131072, 131072, 0), (60000, 20, 131072, 131072, 1),
    (60000, 1, 131072, 131072, 1), (60000, 1, 131072, 131072, 0)])
def test_the_workspace_has_bounds(lib, B, q_len, own, prefix, dtype):
    for groups in (1, B):
        assert serving(lib, B, q_len, own, prefix, groups=groups, dtype=dtype) <= 512 << 20
        # (splits that are asked for may make one sequence's states more, beside the groups' six words each)
        alone = serving(lib, 1, q_len, own, prefix, dtype=dtype, split_tokens=2048) + 256 + 24 * (B + 1)
        assert serving(lib, B, q_len, own, prefix, groups=groups, dtype=dtype, split_tokens=2048) <= max(512 << 20, alone)
    # a batch that fits is not cut: the bound changes nothing there
    assert serving(lib, 4, 20, own, prefix, dtype=dtype) < 512 << 20


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,q_len,own,prefix,heads", [
    (256, 1024, 1024, 1000, (32, 8)), (2049, 128, 1024, 1000, (32, 8)), (9000, 40, 4096, 40000, (8, 8)),
    (70000, 1, 512, 4000, (8, 8)), (70000, 3, 512, 64, (32, 8))])
def test_batches_of_any_number_of_tiles(lib, B, q_len, own, prefix, heads, dtype):
    for flags in (0, atlas.DEBUG_SHARED_SPLIT, atlas.DEBUG_SHARED_TC, atlas.DEBUG_SHARED_WHOLE):
        for groups in (1, 1 + B // 3, B):
            assert serving(lib, B, q_len, own, prefix, heads, groups, dtype, debug_flags=flags) != SIZE_MAX


@pytest.mark.parametrize("sms", [0, 1, 8, 152, 300])
def test_batches_behind_wide_tables(lib, sms):
    """A line of many tiles of many blocks, whatever the number of SMs that it is cut among."""
    assert serving(lib, 256, 512, 131072, 131072, sm_count=sms) != SIZE_MAX
    assert serving(lib, 64, 1024, 131072, 131072, groups=64, sm_count=sms) != SIZE_MAX


@pytest.mark.parametrize("sms", [0, 1, 8, 152, 300])
def test_the_workspace_is_that_of_the_sms_planned_for(lib, sms):
    """64 steps behind 32768 keys: more SMs, more states."""
    S = prefixes(n_groups=1, max_prefix_pages=2048)
    n = ws(lib, S, Hq=32, Hkv=8, batch=64, max_pages_per_seq=128, sm_count=sms)
    assert atlas.shared_workspace_size((64, 32, 1, 128), 32, 8, 128, 16, 128, 1, 2048, 64, sm_count=sms) == n
    assert sms in (0, 152) or n != ws(lib, S, Hq=32, Hkv=8, batch=64, max_pages_per_seq=128, sm_count=152)


def test_arguments_are_checked_before_any_launch(lib):
    need = ws(lib)
    good = dict(workspace=0x1000, workspace_bytes=need)
    assert call(lib, None, launch(**good)) == 1 and call(lib, prefixes(), None) == 1
    for name in ("prefix_table", "prefix_lens", "group_starts"):
        assert call(lib, prefixes(**{name: None}), launch(**good)) == 1
        assert call(lib, prefixes(**{name: 0x1002}), launch(**good)) == 1
    for k in range(5):
        assert call(lib, prefixes(), launch(**good), tuple(None if j == k else 0x1000 for j in range(5))) == 1
    for k in range(3):
        assert call(lib, prefixes(), launch(**good), tuple(0x1008 if j == k else 0x1000 for j in range(5))) == 1
    assert call(lib, prefixes(), launch(**good, lse=0x1001)) == 1
    assert call(lib, prefixes(), launch(**{**good, "out": None})) == 1
    assert call(lib, prefixes(), launch(**{**good, "out": 0x1008})) == 1
    assert call(lib, prefixes(), launch(workspace=0x1000, workspace_bytes=need - 1)) == 3
    assert call(lib, prefixes(), launch()) == 3
    assert call(lib, prefixes(), launch(workspace=0x1008, workspace_bytes=need)) == 1
    for scale in (float("inf"), float("nan"), -float("inf")):
        assert call(lib, prefixes(), launch(**good), scale=scale) == 1
    assert call(lib, prefixes(), launch(**good, softcap=-1.0)) == 1
    assert call(lib, prefixes(), launch(**good, softcap=float("inf"))) == 1
    assert call(lib, prefixes(), launch(**good, window=3)) == 1
    assert call(lib, prefixes(), launch(**good, phase=1)) == 2


def test_the_plain_form_on_a_case_worked_by_hand():
    # prefix scores 0, ln 2 over values 1, 2; own score ln 3 over 3: weights 1/6, 2/6, 3/6
    pk, pv = np.array([0.0, np.log(2)]).reshape(1, 2, 1), np.array([1.0, 2.0]).reshape(1, 2, 1)
    k, v = np.full((2, 1, 1, 1), np.log(3)), np.full((2, 1, 1, 1), 3.0)
    out, lse = shared_rows(np.ones((2, 2, 1, 1)), [(pk, pv)], [0, 1], k, v, [1, 1], 1.0)
    assert np.allclose(out[0], 14 / 6) and np.allclose(lse[0], np.log(6))
    assert np.allclose(out[1], 3) and np.allclose(lse[1], np.log(3))    # in no group


# ------------------------------------------------------------------ on the GPU
class Case:
    """Random inputs of a call; pages of own caches and prefixes mixed in one pool, everything
    behind their ends NaN, table entries behind them out of range."""

    def __init__(self, dtype, Hq, Hkv, D, P, q_len, starts, pre, lens, seed, ragged=None):
        r = np.random.default_rng(seed)

        def normal(*shape):
            return torch.from_numpy(r.standard_normal(shape, dtype=np.float32)).to(DT[dtype])

        B, n = len(lens), len(pre)
        self.q = normal(B, Hq, q_len, D)
        T = max(list(lens) + list(pre) + [1])
        self.k, self.v = normal(B + n, Hkv, T, D), normal(B + n, Hkv, T, D)
        kp, vp, table = page_kv(self.k.float().numpy(), self.v.float().numpy(), list(lens) + list(pre),
                                P, seed=seed, pad_page=10 ** 6, extra_pages=2)
        width = [max(1, -(-max(x) // P)) for x in (lens, pre)]
        self.sizes = Hq, Hkv, D, P
        self.lens, self.pre, self.starts, self.ragged = list(lens), list(pre), list(starts), ragged
        i32 = dict(dtype=torch.int32, device="cuda")
        self.args = [self.q.cuda(), *(torch.from_numpy(x).to(DT[dtype]).cuda() for x in (kp, vp)),
                     torch.from_numpy(table[B:, : width[1]].copy()).cuda(), torch.tensor(self.pre, **i32),
                     torch.tensor(self.starts, **i32), torch.from_numpy(table[:B, : width[0]].copy()).cuda(),
                     torch.tensor(self.lens, **i32)]
        self.q_lens = None if ragged is None else torch.tensor(ragged, **i32)

    def __call__(self, scale, **kw):
        return atlas.shared(*self.args, *self.sizes, scale, q_lens=self.q_lens, **kw)

    def expected(self, scale, sinks=None, softcap=0.0):
        B = len(self.lens)
        k, v = widen(self.k), widen(self.v)
        parts = [(k[B + n, :, : self.pre[n]], v[B + n, :, : self.pre[n]]) for n in range(len(self.pre))]
        return shared_rows(widen(self.q), parts, self.starts, k[:B], v[:B], self.lens, scale,
                           self.ragged, sinks, softcap)


CASES = [
    # dtype, Hq, Hkv, D, P, q_len, starts, prefix lengths, own lengths, options
    ("bf16", 8, 2, 128, 16, 1, [0, 3], [300], [1, 17, 40], {}),
    ("bf16", 8, 2, 128, 16, 1, [0, 1], [1], [1], {}),                              # one key and one key
    ("bf16", 4, 4, 64, 64, 1, [0, 2, 5], [129, 1000], [1, 64, 65, 3, 200], dict(sinks=True)),
    ("bf16", 8, 1, 128, 8, 1, [0, 20], [700], list(range(1, 21)), {}),             # 160 rows: a pair of tiles
    ("bf16", 8, 2, 64, 16, 3, [0, 0, 4, 4], [50, 77, 5], [3, 4, 60, 9], {}),        # empty groups
    ("bf16", 4, 2, 128, 32, 1, [1, 3], [90], [5, 6, 7, 8], {}),                    # some in no group
    ("bf16", 6, 2, 64, 16, 5, [0, 2, 4], [0, 260], [5, 9, 30, 77], dict(ragged=[5, 1, 0, 3])),
    ("bf16", 12, 4, 128, 128, 2, [0, 1, 2, 3], [128, 127, 129], [2, 128, 300], dict(softcap=3.0, scale=-0.07)),
    ("bf16", 8, 2, 128, 16, 40, [0, 3], [513], [40, 41, 90], {}),                  # 480 rows, own tiles too
    ("bf16", 4, 1, 64, 64, 150, [0, 2, 3], [200, 64], [150, 333, 151], dict(ragged=[150, 9, 131])),
    ("bf16", 8, 2, 128, 16, 1, [0, 40], [1025], [1 + 5 * b % 33 for b in range(40)], dict(split_tokens=64)),
    ("bf16", 16, 2, 128, 16, 1, [0, 2], [3000], [100, 2], dict(split_tokens=128, sinks=True)),
    ("bf16", 2, 1, 64, 16, 1, list(range(0, 41)), [3 * n % 50 for n in range(40)], [1 + n % 7 for n in range(40)], {}),
    ("f32", 8, 2, 128, 16, 1, [0, 3], [300], [1, 17, 40], {}),
    ("f32", 4, 4, 64, 32, 1, [0, 1, 4], [1, 1000], [1, 64, 65, 3], dict(sinks=True)),
    ("f32", 8, 1, 64, 8, 2, [0, 20], [700], list(range(2, 22)), {}),               # three tiles
    ("f32", 6, 2, 128, 16, 5, [0, 2, 4], [0, 260], [5, 9, 30, 77], dict(ragged=[5, 1, 0, 3])),
    ("f32", 4, 2, 64, 128, 33, [0, 1, 2], [129, 65], [33, 300], dict(softcap=4.0, scale=-0.11)),
    ("f32", 8, 2, 128, 64, 1, [1, 2], [2100], [5, 70], dict(split_tokens=192)),
    # more tiles than a CTA each: pieces that go on, are cut, and are whole
    ("bf16", 8, 2, 128, 16, 1, [0, 30, 33, 64], [9000, 700, 3100], [1 + 7 * b % 90 for b in range(64)], {}),
    ("bf16", 8, 8, 64, 64, 3, [0, 1, 100], [2000, 5000], [3 + b % 70 for b in range(100)], dict(ragged=[b % 4 for b in range(100)])),
    ("bf16", 4, 2, 128, 32, 130, [0, 3, 5], [3000, 129], [130, 200, 700, 131, 2000], dict(sinks=True)),
    ("bf16", 8, 8, 128, 16, 64, [0, 12], [4500], [64 + 9 * b for b in range(12)], dict(ragged=[64 - 5 * b for b in range(12)])),
    ("bf16", 2, 2, 64, 8, 300, [0, 1, 2], [640, 9], [300, 411], dict(softcap=6.0)),
    ("bf16", 40, 40, 64, 16, 1, list(range(0, 71, 2)), [1 + n % 3 for n in range(35)], [1 + b % 3 for b in range(70)], {}),
    # own keys of 17 to 32 rows as splits beside the tiles
    ("bf16", 8, 2, 128, 16, 7, [0, 3, 5], [300, 41], [7, 40, 200, 9, 1000], dict(ragged=[7, 0, 3, 7, 1])),
    ("bf16", 8, 1, 64, 32, 4, [0, 30], [900], list(range(4, 34)), dict(sinks=True)),
    # more tiles than the pieces of one wave of CTAs
    ("bf16", 64, 64, 64, 16, 1, [0, 100, 200], [130, 1], [1 + b % 5 for b in range(200)], {}),
]


def check(x, dtype, scale, **opt):
    sinks = torch.linspace(-1, 3, x.sizes[0]) if opt.get("sinks") else None
    ref, ref_lse = x.expected(scale, None if sinks is None else widen(sinks), opt.get("softcap", 0.0))
    kw = dict(split_tokens=opt.get("split_tokens", 0), softcap=opt.get("softcap", 0.0),
              debug_flags=opt.get("path", 0), sinks=None if sinks is None else sinks.cuda())
    out = torch.full(x.q.shape, 99.0, dtype=torch.float32, device="cuda")
    lse = torch.full(x.q.shape[:3], 99.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert x(scale, out=out, lse=lse, status=status, **kw) is out
    assert int(status.item()) == 0
    got, got_lse = widen(out), widen(lse)
    real = ~np.isnan(ref_lse)
    assert (got[~real] == 99).all() and (got_lse[~real] == 99).all()   # padding rows stay
    assert np.isfinite(got).all()
    tol = F32_REL * np.abs(ref[real]).max() if dtype == "f32" else BF16_ABS
    assert np.abs(got[real] - ref[real]).max() <= tol
    assert np.abs(got_lse[real] - ref_lse[real]).max() <= (2e-5 if dtype == "f32" else 1e-4)
    if dtype == "bf16":                                                # the bf16 output rounds it
        low = torch.full(x.q.shape, 99.0, dtype=torch.bfloat16, device="cuda")
        x(scale, out=low, **kw)
        assert torch.equal(low, out.to(torch.bfloat16))


@gpu
@pytest.mark.parametrize("path", [0, atlas.DEBUG_SHARED_SPLIT, atlas.DEBUG_SHARED_TC,
                                  atlas.DEBUG_SHARED_WHOLE | atlas.DEBUG_SHARED_TC])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,P,q_len,starts,pre,lens,opt", CASES)
def test_matches_the_plain_form(dtype, Hq, Hkv, D, P, q_len, starts, pre, lens, opt, path):
    x = Case(dtype, Hq, Hkv, D, P, q_len, starts, pre, lens, 200 + q_len, opt.get("ragged"))
    check(x, dtype, **{"scale": D ** -0.5, **opt}, path=path)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,q_len", [(5, 1), (3, 24)])
def test_no_prefix_is_a_suffix(dtype, B, q_len):
    """Prefixes of no keys leave the states of the sequences' own splits: with the same split
    size the merge gives the suffix call's bits.  fp32 rows of more than 16 take products of the
    more exact form: both calls are within F32_REL of the largest of the same exact rows, so within
    twice that of one another."""
    lens = [q_len + 31 * b for b in range(B)]
    x = Case(dtype, 8, 2, 128, 16, q_len, [0, 2, B], [0, 0], lens, 3)
    a = x(0.09, split_tokens=64)
    q, kp, vp, _, _, _, table, own = x.args
    b = atlas.suffix(q, kp, vp, table, own, *x.sizes, 0.09, split_tokens=64)
    if dtype == "f32" and q_len > 4:
        assert float((a - b).abs().max()) <= 2 * F32_REL * float(b.abs().max()) * (1 + F32_REL)
    else:
        assert torch.equal(a, b)


@gpu
def test_the_order_of_the_groups_changes_no_bits():
    """On the split kernels a sequence's result depends on its own group alone."""
    x = Case("bf16", 8, 2, 128, 16, 1, [0, 2, 5], [300, 90], [9, 8, 7, 6, 5], 4)
    a = x(0.09)
    q, kp, vp, ptab, plen, starts, table, own = x.args
    at = torch.tensor([2, 3, 4, 0, 1], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    b = atlas.shared(q[at].contiguous(), kp, vp, ptab.flip(0).contiguous(), plen.flip(0).contiguous(),
                     torch.tensor([0, 3, 5], **i32), table[at].contiguous(), own[at].contiguous(), *x.sizes, 0.09)
    assert torch.equal(a[at], b)


@gpu
@pytest.mark.parametrize("dtype,q_len,path", [("bf16", 1, 4), ("bf16", 1, 8), ("bf16", 1, 24), ("bf16", 40, 8),
                                              ("bf16", 40, 16), ("f32", 1, 4), ("f32", 1, 8), ("f32", 40, 0)])
def test_bad_lengths_groups_and_pages_are_reported(dtype, q_len, path):
    x = Case(dtype, 8, 2, 64, 16, q_len, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8)
    good = x(0.1, debug_flags=path)

    def again(k, value, bit, nan):
        args = list(x.args)
        args[k] = torch.tensor(value, dtype=torch.int32, device="cuda") if isinstance(value, list) else value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = atlas.shared(*args, *x.sizes, 0.1, status=status, debug_flags=path)
        assert int(status.item()) == bit
        for b in range(4):
            if b in nan:
                assert torch.isnan(out[b]).all()
            elif dtype == "bf16" and path != atlas.DEBUG_SHARED_SPLIT:
                # the tiles are cut elsewhere when a sequence drops out: both results are within
                # the bound of the same exact rows, |out| <= 4 here, so twice that apart at most
                assert float((out[b].float() - good[b].float()).abs().max()) <= 2 * (BF16_ABS + 2.0 ** -8 * 4)
            else:
                assert torch.equal(out[b], good[b])

    assert float(good.float().abs().max()) <= 4
    for bad in (-1, x.args[3].shape[1] * 16 + 1):
        again(4, [100, bad], atlas.DEV_BAD_SEQLEN, (2, 3))
    for bad in (q_len - 1, x.args[6].shape[1] * 16 + 1):
        again(7, [50, bad, 60, 77], atlas.DEV_BAD_SEQLEN, (1,))
    for starts in ([-1, 2, 4], [0, 2, 5], [2, 0, 4], [0, 4, 2], [0, 2 ** 31 - 1, 4], [0, -(2 ** 31), 4]):
        again(5, starts, atlas.DEV_BAD_SEQLEN, (0, 1, 2, 3))
    for k, row, nan in ((3, 0, (0, 1)), (6, 3, (3,))):
        for page in (-5, x.args[1].shape[0]):
            table = x.args[k].clone()
            table[row, 1] = page
            again(k, table, atlas.DEV_BAD_PAGE, nan)


@gpu
@pytest.mark.parametrize("path", [0, 4, 8, 24])
@pytest.mark.parametrize("dtype,q_len", [("bf16", 3), ("bf16", 40), ("f32", 3), ("f32", 24)])
def test_bad_query_counts_are_reported(dtype, q_len, path):
    x = Case(dtype, 8, 2, 64, 16, q_len, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8, [q_len, 2, q_len, 1])
    good = x(0.1, debug_flags=path, out=torch.zeros_like(x.args[0]))
    for bad in (-1, q_len + 1, 2 ** 31 - 1, -(2 ** 31)):
        x.q_lens = torch.tensor([q_len, bad, q_len, 1], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = x(0.1, status=status, debug_flags=path, out=torch.zeros_like(x.args[0]))
        assert int(status.item()) == atlas.DEV_BAD_SEQLEN
        assert torch.isnan(out[1]).all()
        for b in (0, 2, 3):   # (twice the bound, as for bad lengths)
            tol = 2 * (BF16_ABS + 2.0 ** -8 * 4) if dtype == "bf16" else 2 * F32_REL * 4
            assert float((out[b].float() - good[b].float()).abs().max()) <= tol


@gpu
@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("bf16", 24), ("f32", 1)])
def test_captured_and_replayed_with_other_groups_and_lengths(dtype, q_len):
    x = Case(dtype, 8, 2, 128, 16, q_len, [0, 2, 4], [500, 100], [40, 41, 60, 77], 9)
    q, kp, vp, ptab, plen, starts, table, own = x.args
    out = torch.empty_like(q)
    space = torch.empty(atlas.shared_workspace_size(q.shape, 8, 2, 128, 16, table.shape[1], 2, ptab.shape[1],
                                                    kp.shape[0], dtype=DT[dtype]),
                        dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        x(0.09, out=out, workspace=space)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            x(0.09, out=out, workspace=space)
    for p, s, o in (([500, 100], [0, 2, 4], [40, 41, 60, 77]), ([0, 100], [0, 3, 4], [24, 33, 25, 70]),
                    ([1, 0], [4, 4, 4], [40, 30, 24, 25])):
        torch.cuda.synchronize()
        for t, value in ((plen, p), (starts, s), (own, o)):
            t.copy_(torch.tensor(value, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, x(0.09))


PATHS = [0, atlas.DEBUG_SHARED_SPLIT, atlas.DEBUG_SHARED_TC, atlas.DEBUG_SHARED_WHOLE | atlas.DEBUG_SHARED_TC]


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,Hq,Hkv,D,q_len,ragged", [
    ("bf16", 2, 1, 64, 1, False), ("bf16", 2, 1, 128, 3, True), ("f32", 2, 1, 64, 2, True)])
def test_more_sequences_and_groups_than_the_plan_has_threads(dtype, Hq, Hkv, D, q_len, ragged, path):
    """1300 sequences in 601 groups: of none, of one, of few, and one of 600; some in none."""
    starts = [0, 0, 600] + [600 + min(n, 500) for n in range(1, 598)] + [1200, 1290]
    pre = [(0, 40, 130, 7)[n % 4] for n in range(len(starts) - 1)]
    pre[1] = 300
    lens = [q_len + b * 7 % 40 for b in range(1300)]
    x = Case(dtype, Hq, Hkv, D, 8, q_len, starts, pre, lens, 17,
             [b % (q_len + 1) for b in range(1300)] if ragged else None)
    check(x, dtype, D ** -0.5, path=path)


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_query_at_all(dtype, path):
    x = Case(dtype, 8, 2, 64, 16, 3, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8, [0, 0, 0, 0])
    out = torch.full_like(x.args[0], 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x(0.1, out=out, status=status, debug_flags=path)
    assert (out == 7).all() and int(status.item()) == 0


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_pages_twice(dtype, path):
    """Two groups behind the same prompt, and a sequence whose own pages are a prefix's too."""
    x = Case(dtype, 8, 2, 64, 16, 1, [0, 2, 4], [300, 300], [50, 41, 60, 300], 12)
    x.args[3][1] = x.args[3][0]
    x.args[6][3] = x.args[3][0]
    for t in (x.k, x.v):
        t[5] = t[4]
        t[3] = t[4]
    check(x, dtype, 0.125, path=path)


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,D,q_len", [("bf16", 128, 1), ("bf16", 64, 40), ("f32", 128, 1)])
def test_pages_whose_offsets_pass_32_bits(dtype, D, q_len, path):
    """The same pages at the end of a pool of more than 2^32 elements."""
    x = Case(dtype, 4, 2, D, 128, q_len, [0, 2, 3], [300, 129], [50, 141, 260], 12)
    q, kp, vp, ptab, plen, starts, table, own = x.args
    near = x(0.1, debug_flags=path)
    n = kp.shape[0]
    num = (1 << 32) // (2 * 128 * D) + 2 * n
    far = [torch.empty((num, *kp.shape[1:]), dtype=kp.dtype, device="cuda") for _ in range(2)]
    for a, b in zip(far, (kp, vp)):
        a[num - n:] = b
    moved = [torch.where(t < n, t + (num - n), t) for t in (ptab, table)]
    out = atlas.shared(q, *far, moved[0], plen, starts, moved[1], own, *x.sizes, 0.1, debug_flags=path)
    assert torch.equal(out, near)


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("bf16", 40), ("f32", 2)])
def test_calls_on_two_streams_at_once(dtype, q_len, path):
    """Each with its own workspace: the bits are those of calls one after the other."""
    x = [Case(dtype, 8, 2, 128, 16, q_len, [0, 30, 40], [2000, 300], [q_len + b for b in range(40)], s) for s in (1, 2)]
    want = [c(0.09, debug_flags=path) for c in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for c, s, g in zip(x, streams, got):
            with torch.cuda.stream(s):
                g.append(c(0.09, debug_flags=path))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, y) for y in g)


@gpu
@pytest.mark.parametrize("prefix,B,path,least", [(32768, 32, 8, 137), (8192, 32, 8, 132), (8192, 64, 8, 132),
                                                 (8192, 1, 24, 137)])
def test_the_line_is_cut_among_all_sms(prefix, B, path, least):
    """8 kv heads behind long prefixes with next to no own keys: the shares (in the plan's record of
    a sequence, or of whole tiles the numbers of pieces) leave a tenth of the SMs without work at most.
    (Where a tile's 64 blocks have room for 64 / 4 + 3 states, and are cut in 17 at most, a share has 4
    of the 66 that each of 8 tiles counts for: 132.)"""
    n, G, Hkv, P, D = (1, 4, 8, 64, 64) if path == 8 else (30, 4, 8, 64, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = prefix // P
    q = torch.randn(B, G * Hkv, n, D, device="cuda").to(torch.bfloat16)
    kp, vp = (torch.randn(pages + B, Hkv, P, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    space = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    atlas.shared(q, kp, vp, torch.arange(pages, **i32)[None], torch.tensor([prefix], **i32),
                 torch.tensor([0, B], **i32), torch.arange(pages, pages + B, **i32)[:, None],
                 torch.full((B,), n, **i32), G * Hkv, Hkv, D, P, 0.1, workspace=space, debug_flags=path, sm_count=152)
    words = space.view(torch.int32)
    if path == 8:
        # a sequence's record: blocks, rows before it, rows, first place, length of a head, weight, share
        at = ((words[:-8] == prefix // 128) & (words[1:-7] == 0) & (words[2:-6] == B * G * n) &
              (words[3:-5] == 0)).nonzero().flatten().tolist()
        assert len(at) == 1
        line, share = int(words[at[0] + 4]) * Hkv, int(words[at[0] + 6])
        ctas = -(-line // share)
    else:
        # a CTA's piece of whole tiles: unit, kv head, first row, rows, first block, blocks, state, keys, own keys
        ctas = int(((words[3:-6] == G * n) & (words[7:-2] == prefix) & (words[8:-1] == n)).sum()) - (Hkv - 1)
    assert least <= ctas <= 153


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fewer_sms_and_events(dtype, path):
    x = Case(dtype, 8, 2, 128, 16, 1, [0, 30, 40], [2000, 300], [1 + b for b in range(40)], 5)
    ref, _ = x.expected(0.09)
    timer = atlas.EventTimer()
    tol = F32_REL * np.abs(ref).max() if dtype == "f32" else BF16_ABS
    for sms in (1, 7, 1000):
        out = x(0.09, debug_flags=path, sm_count=sms, events=timer.handles, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert np.abs(widen(out) - ref).max() <= tol
        assert timer.main_ms() > 0 and timer.merge_ms() > 0


@gpu
@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype,q_len", [("bf16", 1), ("bf16", 40), ("f32", 1), ("f32", 24)])
def test_a_workspace_of_the_size_given_for_that_many_sms(dtype, q_len, path):
    x = Case(dtype, 8, 2, 128, 16, q_len, [0, 30, 40], [2000, 300], [q_len + b for b in range(40)], 5)
    q, kp, _, ptab, _, starts, table, _ = x.args
    for sms in (1, 7, 152, 300):
        n = atlas.shared_workspace_size(q.shape, *x.sizes, table.shape[1], len(starts) - 1, ptab.shape[1],
                                        kp.shape[0], dtype=DT[dtype], debug_flags=path, sm_count=sms)
        space = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
        want = x(0.09, debug_flags=path, sm_count=sms)
        assert torch.equal(x(0.09, debug_flags=path, sm_count=sms, workspace=space[:n]), want)
        assert (space[n:] == 77).all()
        with pytest.raises(atlas.AtlasError):
            x(0.09, debug_flags=path, sm_count=sms, workspace=space[:n - 1])


def test_tensors_on_the_host():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        atlas.shared(torch.ones(2, 8, 1, 64), torch.ones(4, 2, 16, 64), torch.ones(4, 2, 16, 64),
                     torch.zeros((1, 1), **i32), torch.zeros(1, **i32), torch.zeros(2, **i32),
                     torch.zeros((2, 1), **i32), torch.ones(2, **i32), 8, 2, 64, 16, 0.1)


def apart(t):
    """The same shape and values, not contiguous."""
    return torch.stack([t, t], -1)[..., 0]


NAMES = ["q", "k_pages", "v_pages", "prefix_table", "prefix_lens", "group_starts", "page_table", "seq_lens"]
BAD = [(n, f) for n in NAMES for f in (apart, torch.Tensor.cpu, torch.Tensor.double, lambda t: t[:1])] + [
    ("q", lambda t: t[:, :4].contiguous()), ("q", lambda t: t[0]), ("k_pages", lambda t: t[:, :1].contiguous()),
    ("group_starts", lambda t: t[:-1]), ("prefix_table", lambda t: t[0]), ("page_table", lambda t: t[0])]


@gpu
@pytest.mark.parametrize("k", range(len(BAD)), ids=[f"{n}{i}" for i, (n, _) in enumerate(BAD)])
def test_one_wrong_tensor(k):
    x = Case("bf16", 8, 2, 64, 16, 2, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8)
    name, change = BAD[k]
    at = NAMES.index(name)
    out, lse = torch.zeros_like(x.args[0]), torch.zeros(x.q.shape[:3], device="cuda")
    x.args[at] = change(x.args[at])
    with pytest.raises(ValueError):
        x(0.1, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == 0).all()


@gpu
@pytest.mark.parametrize("name,make", [
    ("out", lambda: torch.zeros(4, 8, 1, 64, device="cuda", dtype=torch.bfloat16)),
    ("out", lambda: torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16)),
    ("lse", lambda: torch.zeros(4, 8, 1, device="cuda")), ("lse", lambda: torch.zeros(4, 8, 2, device="cuda").double()),
    ("status", lambda: torch.zeros(0, dtype=torch.int32, device="cuda")),
    ("sinks", lambda: torch.zeros(2, device="cuda")), ("sinks", lambda: torch.zeros(8)),
    ("workspace", lambda: torch.zeros(1 << 22, dtype=torch.uint8))])
def test_one_wrong_option(name, make):
    x = Case("bf16", 8, 2, 64, 16, 2, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8)
    with pytest.raises(ValueError):
        x(0.1, **{name: make()})
    with pytest.raises(atlas.AtlasError):
        x(0.1, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


@gpu
@pytest.mark.parametrize("path", PATHS)
def test_outputs_over_inputs(path):
    x = Case("bf16", 8, 2, 64, 16, 2, [0, 2, 4], [100, 70], [50, 41, 60, 77], 8)
    before = [t.clone() for t in x.args[:3]]
    space = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    rows = x.q.shape[0] * 8 * 2
    over = [dict(out=x.args[0]), dict(out=x.args[1].reshape(-1)[:rows * 64].reshape(x.q.shape)),
            dict(out=x.args[2].reshape(-1)[-rows * 64:].reshape(x.q.shape)), dict(workspace=x.args[0]),
            dict(workspace=space, out=space[1024:1024 + rows * 128].view(torch.bfloat16).reshape(x.q.shape)),
            dict(workspace=space, lse=space[4096:4096 + rows * 4].view(torch.float32).reshape(x.q.shape[:3])),
            dict(out=space[:rows * 128].view(torch.bfloat16).reshape(x.q.shape),
                 lse=space[16:16 + rows * 4].view(torch.float32).reshape(x.q.shape[:3]))]
    for kw in over:
        with pytest.raises(atlas.AtlasError):
            x(0.1, debug_flags=path, **kw)
    torch.cuda.synchronize()
    bits = [[y.view(torch.int16) for y in z] for z in (before, x.args[:3])]       # (they hold NaN)
    assert all(torch.equal(a, b) for a, b in zip(*bits)) and (space == 0).all()
    # side by side they are accepted
    out = space[:rows * 128].view(torch.bfloat16).reshape(x.q.shape)
    lse = space[rows * 128:rows * 132].view(torch.float32).reshape(x.q.shape[:3])
    assert torch.equal(x(0.1, debug_flags=path, out=out, lse=lse, workspace=space[rows * 132:]),
                       x(0.1, debug_flags=path))
