"""Keys that hold infinities or NaN, in every kernel of atlas_kv_weights: the weights of the
other keys keep their bits, a key that no row sees gets 0 whatever it holds, and a key's own
weight is the plain form's (exp of its scores: 0, infinite or NaN) or, where the scores are
sums of tf32 parts (fp32 with more than two rows per kv head), NaN."""
import math

import numpy as np
import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.operator_refs import key_weights, row_lse, widen
from tests.paging import page_kv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = math.inf, math.nan

CASES = [
    # dtype, Hq, Hkv, D, q_len, options                       kernel
    ("bf16", 8, 2, 128, 1, {}),                             # stream, 16 columns
    ("bf16", 8, 2, 64, 7, dict(softcap=5.0)),               # 32
    ("bf16", 8, 2, 128, 16, dict(window=90)),               # 64
    ("bf16", 4, 1, 64, 50, {}),                             # 256
    ("bf16", 4, 2, 128, 300, {}),                           # tiles
    ("bf16", 4, 2, 64, 300, dict(window=90)),
    ("f32", 2, 2, 128, 1, {}),                              # by warps, one column
    ("f32", 4, 2, 64, 1, dict(window=90)),                  # two
    ("f32", 2, 2, 128, 2, dict(softcap=5.0)),
    ("f32", 8, 2, 128, 3, {}),                              # tf32 parts, stream
    ("f32", 8, 2, 64, 16, dict(window=90)),
    ("f32", 8, 2, 128, 40, dict(sm_count=1)),               # in three launches
    ("f32", 8, 2, 128, 40, {}),                             # tiles
    ("f32", 4, 1, 64, 200, dict(window=90)),
]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,q_len,opt", CASES)
def test_nonfinite_keys(dtype, Hq, Hkv, D, q_len, opt):
    P, lens, scale = 16, [q_len + 400, q_len + 133], D ** -0.5
    r = np.random.default_rng(D + q_len)
    q, k = (torch.from_numpy(r.standard_normal(s, dtype=np.float32)).to(DT[dtype])
            for s in ((2, Hq, q_len, D), (2, Hkv, max(lens), D)))
    var = dict(window=opt.get("window", 0), softcap=opt.get("softcap", 0.0))
    lse = np.float32(row_lse(widen(q), widen(k), lens, scale, **var))
    bad = k.clone()
    # one element of a row (scores of either sign or, with -0, none), whole rows, and rows in
    # the first tile, at its border, in the last rows' own positions and at the end
    rows = [(3, slice(5, 6), INF), (4, slice(5, 6), -INF), (17, slice(0, D), INF), (40, slice(0, D), NAN),
            (127, slice(D - 1, D), -INF), (128, slice(0, 1), NAN), (lens[1] - 1, slice(1, 2), INF),
            (lens[1] - q_len, slice(2, 3), -INF), (300, slice(0, 1), -INF)]
    for t, at, x in rows:
        bad[:, :, t, at] = x
    touched = np.zeros(max(lens), bool)
    touched[[t for t, _, _ in rows]] = True

    def weights(keys):
        kp, _, table = page_kv(keys.float().numpy(), keys.float().numpy(), lens, P, seed=3)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = atlas.kv_weights(q.cuda(), torch.from_numpy(kp).to(DT[dtype]).cuda(), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(lse).cuda(),
                             Hq, Hkv, D, P, scale, accumulate=False, status=status,
                             sm_count=opt.get("sm_count", 0), **var)
        assert int(status.item()) == 0
        return w.cpu()

    got, finite = weights(bad), weights(k)
    with np.errstate(all="ignore"):
        want = key_weights(widen(q), widen(bad), lens, lse.astype(np.float64), scale, **var)
    parts = dtype == "f32" and Hq // Hkv * q_len > 2
    for b, L in enumerate(lens):
        other = ~touched[:L]
        assert torch.equal(got[b, :, :L][:, other], finite[b, :, :L][:, other])
        unseen = np.arange(L) < (L - q_len + 1 - opt["window"] if "window" in opt else 0)
        assert (got[b, :, :L][:, unseen] == 0).all() and (want[b, :, :L][:, unseen] == 0).all()
        for t in np.flatnonzero(touched[:L] & ~unseen):
            for g in range(Hkv):
                x, y = float(got[b, g, t]), want[b, g, t]
                if math.isnan(x):
                    assert math.isnan(y) or parts, (b, g, t, y)
                else:
                    assert x == y or abs(x - y) <= 2e-5 * y, (b, g, t, x, y)
