"""NaN and infinities behind shared prefixes, on every path of atlas_attn_shared.  They are not scanned
for and propagate, as in the other attention calls: a NaN in a key makes the rows that see it NaN and
leaves every other as it is; one in a value makes its element of them NaN, and an infinite one infinite
or NaN (infinity times a second part of a weight, which may be 0); a key whose score is -inf has no
weight and one whose score is +inf makes the row NaN, as exp(inf - inf) is (every row of its group where
fp32 scores are sums of tf32 parts).  Sinks are scores too.  Tolerances are those of tests/test_shared.py."""
import math

import pytest
import torch

import exact_causal_gqa_gb300 as atlas
from tests.gpu_helpers import BF16_ABS, F32_REL
from tests.test_shared_large import SPLIT, TC, WHOLE, Batch, ints

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan
G = 4
STARTS, PRE = [0, 3, 40, 41], [300, 129, 700]     # (sequences 41 and on in no group)
# dtype, q_len, path; whether the tf32 kernels take the prefixes, and the own keys
PATHS = [("bf16", 1, 0, 0, 0), ("bf16", 1, SPLIT, 0, 0), ("bf16", 1, TC, 0, 0), ("bf16", 1, WHOLE, 0, 0),
         ("bf16", 6, TC, 0, 0), ("bf16", 40, TC, 0, 0), ("bf16", 40, WHOLE, 0, 0), ("bf16", 130, 0, 0, 0),
         ("f32", 1, SPLIT, 0, 0), ("f32", 1, TC, 1, 0), ("f32", 9, 0, 1, 1)]


def batch(dtype, q_len, D=64):
    return Batch(dtype, 2 * G, 2, D, 16, q_len, STARTS, PRE, [q_len + 7 * b % 90 for b in range(44)])


def same(x, path, some, want=None, sinks=None, elements=None):
    """The rows of the sequences `some` are the exact ones; want(b, out, lse) changes what is expected."""
    out, lse = torch.empty(x.q.shape, device="cuda"), torch.empty(x.q.shape[:3], device="cuda")
    status = ints([0])
    x(out=out, lse=lse, status=status, debug_flags=path, sinks=sinks)
    assert int(status.item()) == 0
    f32 = x.q.dtype == torch.float32
    for b in some:
        ref, ref_lse = x.exact(b)
        ref_lse = torch.where(ref_lse == INF, NAN, ref_lse)   # M + ln sum exp(s - M), M = inf
        if want is not None:
            ref, ref_lse = want(b, ref, ref_lse)
        fine = torch.isfinite(ref)
        assert torch.equal(torch.isfinite(out[b]), fine), b
        top = float(ref[fine].abs().max()) if bool(fine.any()) else 0.0
        assert bool(((out[b].double() - ref).abs()[fine] <= (F32_REL * top if f32 else BF16_ABS)).all()), b
        fine = torch.isfinite(ref_lse)
        assert torch.equal(torch.isnan(lse[b]), torch.isnan(ref_lse)), b
        assert bool(((lse[b].double() - ref_lse).abs()[fine] <= (2e-5 if f32 else 1e-4)).all()), b
    return out, lse


SOME = [0, 2, 3, 20, 39, 40, 41, 43]


@pytest.mark.parametrize("dtype,q_len,path,tf32,own_tf32", PATHS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_key_of_a_prefix(dtype, q_len, path, tf32, own_tf32, value):
    for t in (0, 128):
        x = batch(dtype, q_len)
        x.k[int(x.prefix_table[1, t // 16]), 0, t % 16, 5] = value   # kv head 0 of group 1

        def want(b, out, lse):
            if tf32 and 3 <= b < 40:
                out[:G], lse[:G] = NAN, NAN
            return out, lse
        out, _ = same(x, path, SOME, want)
        assert bool(torch.isnan(out[3:40, :G]).any()) and bool(torch.isfinite(out[3:40, G:]).all())
        assert bool(torch.isfinite(out[:3]).all()) and bool(torch.isfinite(out[40:]).all())


@pytest.mark.parametrize("dtype,q_len,path,tf32,own_tf32", PATHS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_an_own_key(dtype, q_len, path, tf32, own_tf32, value):
    """One that the rows from the middle on see."""
    x = batch(dtype, q_len)
    t = x.lens[20] - q_len + q_len // 2
    x.k[int(x.table[20, t // 16]), 1, t % 16, 9] = value

    def want(b, out, lse):
        if own_tf32 and b == 20:
            out[G:, q_len // 2:], lse[G:, q_len // 2:] = NAN, NAN
        return out, lse
    out, _ = same(x, path, SOME, want)
    assert bool(torch.isfinite(out[20, :G]).all()) and bool(torch.isfinite(out[20, :, : q_len // 2]).all())


@pytest.mark.parametrize("dtype,q_len,path,tf32,own_tf32", PATHS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_value(dtype, q_len, path, tf32, own_tf32, value):
    """Of a prefix, and the first of a sequence's own."""
    x = batch(dtype, q_len)
    x.v[int(x.prefix_table[0, 3]), 1, 2, 7] = value
    x.v[int(x.table[20, 0]), 0, 0, 63] = value

    def want(b, out, lse):
        if b < 3:
            out[G:, :, 7] = NAN
        if b == 20:
            out[:G, :, 63] = NAN
        return out, lse
    if q_len > 1:   # (the first own key is one that every row sees)
        assert x.lens[20] > q_len
    out, _ = same(x, path, SOME, want)
    if value == NAN:
        assert bool(torch.isnan(out[:3, G:, :, 7]).all()) and bool(torch.isnan(out[20, :G, :, 63]).all())


@pytest.mark.parametrize("dtype,q_len,path,tf32,own_tf32", PATHS)
def test_no_key_with_a_weight(dtype, q_len, path, tf32, own_tf32):
    """Sequence 40, alone behind a prefix, whose scores are all -inf for kv head 0: the rows are NaN, and
    with sinks 0, of the sink's lse."""
    x = batch(dtype, q_len)
    x.q[40] = x.q[40].abs() + 0.1
    for table, n in ((x.prefix_table[2], 700), (x.table[40], x.lens[40])):
        x.k[table[: -(-n // 16)].long(), 0, :, 3] = -INF
    sinks = torch.linspace(-1, 2, 2 * G, device="cuda")
    for sink in (None, sinks):
        out, lse = (torch.empty(s, device="cuda") for s in (x.q.shape, x.q.shape[:3]))
        x(out=out, lse=lse, debug_flags=path, sinks=sink)
        assert bool(torch.isfinite(out[:40]).all()) and bool(torch.isfinite(out[41:]).all())
        assert bool(torch.isfinite(out[40, G:]).all()) and bool(torch.isfinite(lse[40, G:]).all())
        if sink is None or tf32:
            assert bool(torch.isnan(out[40, :G]).all())
        else:
            assert bool((out[40, :G] == 0).all())
            assert bool(((lse[40, :G] - sinks[:G, None]).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("dtype,q_len,path,tf32,own_tf32", PATHS)
def test_sinks(dtype, q_len, path, tf32, own_tf32):
    """-inf is no sink; NaN and +inf make their heads' rows NaN, as they do a score."""
    x = batch(dtype, q_len)
    sinks = torch.full((2 * G,), -INF, device="cuda")
    same(x, path, SOME, sinks=sinks)
    sinks[1], sinks[6] = NAN, INF

    def want(b, out, lse):
        out[[1, 6]], lse[[1, 6]] = NAN, NAN
        return out, lse
    same(x, path, SOME, want, sinks=sinks)


@pytest.mark.parametrize("dtype,L,split", [("bf16", 513, 512), ("bf16", 513, 64), ("f32", 513, 512), ("f32", 65, 0),
                                           ("f32", 2049, 0), ("bf16", 1, 0), ("bf16", 129, 128), ("f32", 4097, 0)])
@pytest.mark.parametrize("q_len", [1, 2])
def test_a_split_of_one_key_that_is_nan(dtype, L, split, q_len):
    """The same of the split kernels without prefixes: the last key alone in its split."""
    L += q_len - 1
    x = Batch(dtype, 8, 2, 64, 16, q_len, [0, 1], [1], [L, L])
    x.k[int(x.table[1, (L - 1) // 16]), 0, (L - 1) % 16, 2] = NAN
    out = atlas.suffix(x.q, x.k, x.v, x.table, ints(x.lens), *x.sizes, x.scale, split_tokens=split, out_dtype=torch.float32)
    assert bool(torch.isnan(out[1, :G, -1]).all())
    assert bool(torch.isfinite(out[0]).all() & torch.isfinite(out[1, G:]).all() & torch.isfinite(out[1, :, :-1]).all())
    if q_len == 1:
        out = atlas.decode(x.q, x.k, x.v, x.table, ints(x.lens), *x.sizes, x.scale, split_tokens=split)
        assert bool(torch.isnan(out[1, :G]).all()) and bool(torch.isfinite(out[1, G:]).all())
