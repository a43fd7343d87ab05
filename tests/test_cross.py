"""Cross attention (atlas_attn_cross): decoder rows over all of a sequence's encoder
states, against a plain fp64 form; lengths of 0 and 1, ragged rows, every kernel path.

Tolerances are those of the causal calls (gpu_helpers), since the arithmetic is the
same: fp32 1e-5 of the largest |out|, bf16 inputs with fp32 output 2e-3, a bf16 output
the rounding of the fp32 one.  lse: the fp32 form's 2e-5, bf16's 1e-4, as there."""
import ctypes

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from exact_causal_gqa_gb300 import _build
from tests.gpu_helpers import BF16_ABS, F32_REL
from tests.operator_refs import cross_rows, widen
from tests.paging import page_kv

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
    L.batch, L.max_pages_per_seq, L.num_pages, L.q_len = 2, 8, 16, 1
    L.q_dtype = L.kv_dtype = L.out_dtype = 1
    for k, v in kw.items():
        setattr(L, k, v)
    return L


def ws(lib, Hq=8, Hkv=2, D=128, P=16, **kw):
    return lib.atlas_attn_workspace_size(atlas.KIND_CROSS, Hq, Hkv, D, P,
                                         ctypes.byref(launch(**kw)))


@pytest.mark.parametrize("kw", [dict(window=4), dict(window=-1), dict(phase=1), dict(phase=2),
                                dict(chunk_range=0x1000), dict(Hq=7), dict(D=96), dict(P=12),
                                dict(q_len=0), dict(batch=0), dict(q_len=1 << 30),
                                dict(batch=1, Hq=1, Hkv=1, q_len=(1 << 31) - 1)])
def test_cross_refuses(lib, kw):
    assert ws(lib, **kw) == SIZE_MAX


def test_cross_rows_may_outnumber_the_encoder_states(lib):
    assert ws(lib, q_len=1000) != SIZE_MAX      # 128 encoder states at most
    L = launch(q_len=1000)
    assert lib.atlas_attn_workspace_size(atlas.KIND_SUFFIX, 8, 2, 128, 16,
                                         ctypes.byref(L)) == SIZE_MAX


def test_cross_checks_arguments_before_any_launch(lib):
    L = launch(window=4)
    L.out = 0x1000
    args = [0x1000] * 5 + [8, 2, 128, 16, ctypes.c_float(0.1), ctypes.byref(L)]
    assert lib.atlas_attn_cross(*args) == 1      # a window
    L.window, L.phase = 0, 1
    assert lib.atlas_attn_cross(*args) == 2      # a call over several launches
    L.phase = 0
    args[9] = ctypes.c_float(float("inf"))
    assert lib.atlas_attn_cross(*args) == 1
    assert lib.atlas_attn_cross(*([None] * 5 + args[5:])) == 1


def test_the_plain_form_on_a_case_worked_by_hand():
    # scores 0, ln 2, ln 3 over values 1, 2, 3: weights 1/6, 2/6, 3/6
    k = np.array([0.0, np.log(2), np.log(3)]).reshape(1, 1, 3, 1)
    v = np.array([1.0, 2.0, 3.0]).reshape(1, 1, 3, 1)
    out, lse = cross_rows(np.ones((1, 2, 1, 1)), k, v, [3], 1.0)
    assert np.allclose(out, 14 / 6) and np.allclose(lse, np.log(6))
    out, lse = cross_rows(np.ones((1, 1, 1, 1)), k, v, [0], 1.0)
    assert out[0, 0, 0, 0] == 0 and lse[0, 0, 0] == -np.inf
    out, lse = cross_rows(np.ones((1, 1, 1, 1)), k, v, [0], 1.0, sinks=[2.5])
    assert out[0, 0, 0, 0] == 0 and lse[0, 0, 0] == 2.5


# ------------------------------------------------------------------ on the GPU
def problem(dtype, Hq, Hkv, D, P, q_len, lens, seed):
    r = np.random.default_rng(seed)
    T = max(max(lens), 1)
    k = torch.from_numpy(r.standard_normal((len(lens), Hkv, T, D), dtype=np.float32)).to(DT[dtype])
    v = torch.from_numpy(r.standard_normal((len(lens), Hkv, T, D), dtype=np.float32)).to(DT[dtype])
    q = torch.from_numpy(r.standard_normal((len(lens), Hq, q_len, D), dtype=np.float32)).to(DT[dtype])
    kp, vp, table = page_kv(k.float().numpy(), v.float().numpy(), lens, P, seed=seed,
                            pad_page=10 ** 6)
    dev = [torch.from_numpy(x).to(DT[dtype]).cuda() for x in (kp, vp)]
    return q, k, v, [q.cuda(), *dev, torch.from_numpy(table).cuda(),
                     torch.tensor(lens, dtype=torch.int32, device="cuda")]


CASES = [
    # dtype, Hq, Hkv, D, P, q_len, lens, options
    ("bf16", 8, 2, 128, 16, 1, [300, 0, 1, 4097], {}),                    # splits + merge
    ("bf16", 8, 2, 128, 16, 1, [300, 0, 1, 17], {}),                      # one split, direct
    ("bf16", 4, 4, 64, 64, 3, [65, 0, 900], dict(sinks=True)),
    ("bf16", 16, 2, 64, 8, 2, [0, 63, 64, 65], dict(sinks=True, split_tokens=64)),
    ("f32", 4, 4, 64, 16, 1, [512, 0, 1], {}),                            # one cluster per unit
    ("f32", 8, 2, 128, 32, 3, [77, 0, 2000], dict(split_tokens=128)),     # splits + merge
    ("f32", 4, 1, 64, 16, 4, [1, 0, 129], dict(sinks=True)),
    ("bf16", 8, 2, 128, 16, 33, [0, 1, 128, 777], {}),                    # tensor core, splits
    ("bf16", 4, 1, 64, 128, 200, [0, 5, 3001], dict(ragged=[200, 1, 63])),
    ("bf16", 8, 2, 128, 32, 75, [130, 0, 1, 300], dict(direct=True)),     # 3 tiles: a pair and a half
    ("bf16", 6, 2, 64, 16, 128, [257, 0, 64], dict(direct=True, ragged=[128, 7, 0])),
    ("bf16", 8, 1, 128, 64, 128, [129, 0], dict(direct=True, sinks=True, softcap=5.0)),
    ("bf16", 5, 1, 128, 8, 7, [40, 0, 200], dict(direct=True)),           # a single tile
    ("bf16", 8, 2, 128, 16, 33, [200, 0], dict(softcap=3.0, scale=-0.07)),
    ("f32", 8, 2, 128, 16, 33, [0, 1, 64, 777], {}),                      # tf32 products, splits
    ("f32", 4, 1, 64, 32, 130, [0, 65, 300], dict(direct=True, ragged=[130, 0, 31])),
    ("f32", 8, 2, 64, 128, 40, [500, 0], dict(direct=True, sinks=True)),
    # few rows: one launch on long contexts when there are many units, else splits and a merge
    ("bf16", 8, 8, 64, 16, 1, [2000, 0, 1, 700] * 5, {}),
    ("bf16", 16, 8, 128, 64, 2, [1025, 1, 0, 64] * 5, dict(sinks=True, ragged=[2, 1, 2, 0] * 5)),
    ("f32", 4, 4, 64, 16, 1, [3000, 0, 65, 700, 1], {}),
    ("f32", 8, 2, 128, 32, 2, [2048, 0, 1], dict(softcap=4.0)),
    ("f32", 4, 2, 128, 64, 1, [5000, 0, 3], dict(sinks=True)),
    # few tiles on long contexts: automatic splits and the merge
    ("bf16", 4, 1, 128, 16, 40, [3000, 0, 1, 2900], {}),
    ("bf16", 4, 1, 64, 64, 40, [2500, 130, 0], dict(sinks=True, ragged=[40, 3, 0])),
    ("f32", 4, 1, 128, 32, 40, [3000, 0, 1], {}),
    ("f32", 2, 1, 64, 16, 70, [2600, 40, 0], dict(softcap=5.0)),
    # many tiles on short ones: direct
    ("bf16", 8, 8, 128, 32, 300, [300, 0, 41], dict(ragged=[300, 7, 129])),
    ("f32", 8, 8, 64, 32, 130, [130, 200], {}),
]


@gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,D,P,q_len,lens,opt", CASES)
def test_cross_matches_the_plain_form(dtype, Hq, Hkv, D, P, q_len, lens, opt):
    q, k, v, dev = problem(dtype, Hq, Hkv, D, P, q_len, lens, 100 + q_len)
    scale = opt.get("scale", D ** -0.5)
    sinks = torch.linspace(-1, 3, Hq) if opt.get("sinks") else None
    ref, ref_lse = cross_rows(widen(q), widen(k), widen(v), lens, scale, opt.get("ragged"),
                              None if sinks is None else widen(sinks), opt.get("softcap", 0.0))
    kw = dict(split_tokens=opt.get("split_tokens", 0), softcap=opt.get("softcap", 0.0),
              sinks=None if sinks is None else sinks.cuda(),
              debug_flags=atlas.DEBUG_TC_DIRECT if opt.get("direct") else 0,
              q_lens=torch.tensor(opt["ragged"], dtype=torch.int32, device="cuda")
              if "ragged" in opt else None)
    out = torch.full(q.shape, 99.0, dtype=torch.float32, device="cuda")
    lse = torch.full(q.shape[:3], 99.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    atlas.cross(*dev, Hq, Hkv, D, P, scale, out=out, lse=lse, status=status, **kw)
    assert int(status.item()) == 0
    got, got_lse = widen(out), widen(lse)
    real = ~np.isnan(ref_lse)
    assert (got[~real] == 99).all() and (got_lse[~real] == 99).all()   # padding rows stay
    assert np.isfinite(got).all()
    tol = F32_REL * np.abs(ref[real]).max() if dtype == "f32" else BF16_ABS
    assert np.abs(got[real] - ref[real]).max() <= tol
    empty = ref_lse == -np.inf
    assert (got[empty] == 0).all() and (got_lse[empty] == -np.inf).all()
    fine = real & ~empty
    assert np.abs(got_lse[fine] - ref_lse[fine]).max() <= (2e-5 if dtype == "f32" else 1e-4)
    if dtype == "bf16":                                              # the bf16 output rounds it
        low = torch.full(q.shape, 99.0, dtype=torch.bfloat16, device="cuda")
        atlas.cross(*dev, Hq, Hkv, D, P, scale, out=low, **kw)
        assert torch.equal(low, out.to(torch.bfloat16))


@gpu
@pytest.mark.parametrize("dtype,lens", [("bf16", [300, 41, 5000]), ("f32", [512, 17, 2000])])
def test_one_row_is_a_decode(dtype, lens):
    """One query row sees every key either way: the same plan, the same bits."""
    q, k, v, dev = problem(dtype, 8, 2, 128, 16, 1, lens, 7)
    a = atlas.cross(*dev, 8, 2, 128, 16, 0.09)
    assert torch.equal(a, atlas.decode(*dev, 8, 2, 128, 16, 0.09))


@gpu
@pytest.mark.parametrize("dtype,q_len,direct", [("bf16", 1, 0), ("bf16", 40, 0), ("bf16", 40, 1),
                                                ("f32", 1, 0), ("f32", 40, 0), ("f32", 40, 1)])
def test_bad_lengths_and_pages_are_reported(dtype, q_len, direct):
    flags = atlas.DEBUG_TC_DIRECT if direct else 0
    q, k, v, dev = problem(dtype, 8, 2, 64, 16, q_len, [100, 30, 60], 8)
    good = atlas.cross(*dev, 8, 2, 64, 16, 0.1, debug_flags=flags)
    for bad_len in (-1, dev[3].shape[1] * 16 + 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = torch.tensor([100, bad_len, 60], dtype=torch.int32, device="cuda")
        out = atlas.cross(*dev[:4], lens, 8, 2, 64, 16, 0.1, status=status, debug_flags=flags)
        assert int(status.item()) == atlas.DEV_BAD_SEQLEN
        assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    table = dev[3].clone()
    table[1, 1] = -5                             # the second page of 30 states
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = atlas.cross(*dev[:3], table, dev[4], 8, 2, 64, 16, 0.1, status=status, debug_flags=flags)
    assert int(status.item()) == atlas.DEV_BAD_PAGE
    assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


@gpu
def test_cross_is_captured_and_replayed_with_other_lengths():
    q, k, v, dev = problem("bf16", 8, 2, 128, 16, 24, [500, 100], 9)
    out = torch.empty_like(dev[0])
    ws_bytes = atlas.workspace_size("cross", q.shape, 8, 2, 128, 16, dev[3].shape[1],
                                    dev[1].shape[0])
    space = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        atlas.cross(*dev, 8, 2, 128, 16, 0.09, out=out, workspace=space)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            atlas.cross(*dev, 8, 2, 128, 16, 0.09, out=out, workspace=space)
    for lens in ([500, 100], [0, 33]):
        torch.cuda.synchronize()
        dev[4].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, atlas.cross(*dev, 8, 2, 128, 16, 0.09))
