"""How far bf16 attention behind shared prefixes is from fp64 where its outputs are small, over
many keys: a step as atlas_attn_decode's, whatever the number of rows that share the prompt, and the
rows of prompts as those of the library's other tensor-core calls.

A weight as two bf16 parts is off by a half step of the second at most: 2^-8 of what the first
leaves, itself 2^-8 of the weight: 2^-16.  Products of bf16 values accumulate in fp32: at most
2^-23 of sum p |v| for each of 256 products, 2^-15; the scores' rounding is 2e-5 of the weights.
So |out - exact| <= (2^-16 + 2^-15 + 2e-5) sum p |v|.  With one part, the bounds of
tests/test_cross_precision.py: 7.6 * 2^-8 of the root of sum p^2 v^2 on top of that for a single
output, and 2^-8 / sqrt(3) of the outputs' own in the root mean square, 2 % more for the draw."""
import math

import pytest
import torch

import exact_causal_gqa_gb300 as atlas

pytestmark = pytest.mark.gpu
SPLIT, TC, WHOLE = atlas.DEBUG_SHARED_SPLIT, atlas.DEBUG_SHARED_TC, atlas.DEBUG_SHARED_WHOLE | atlas.DEBUG_SHARED_TC
ROUNDING = 2.0 ** -15 + 2e-5  # of sum p |v|, beside the weights'


def call(Hq, Hkv, D, n, B, prefix, own, flags, P=64):
    """The call's rows in fp32, and those of fp64 with sqrt(sum p^2 v^2) and sum p |v|."""
    g = torch.Generator(device="cuda").manual_seed(D + n + B)
    pages, width = -(-prefix // P), -(-own // P)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    q, k, v = normal(B, Hq, n, D), normal(pages + B * width, Hkv, P, D), normal(pages + B * width, Hkv, P, D)
    at = torch.randperm(pages + B * width, generator=g, device="cuda").int()
    table = at[pages:].reshape(B, width)
    out = atlas.shared(q, k, v, at[None, :pages], ints([prefix]), ints([0, B]), table, ints([own] * B), Hq, Hkv,
                       D, P, D ** -0.5, out_dtype=torch.float32, debug_flags=flags)
    seen = torch.arange(prefix + own, device="cuda") <= torch.arange(n, device="cuda")[:, None] + prefix + own - n
    rows = []
    for b in range(B):
        kk, vv = (torch.cat([x[at[:pages].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :prefix],
                             x[table[b].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :own]], 1)
                  .double().repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        p = torch.softmax((q[b].double() @ kk.transpose(1, 2) * D ** -0.5).masked_fill(~seen, -math.inf), -1)
        rows.append((p @ vv, (p ** 2 @ vv ** 2).sqrt(), p @ vv.abs()))
    return out.double(), *(torch.stack(x) for x in zip(*rows))


@pytest.mark.parametrize("flags", [0, SPLIT, TC, WHOLE])
@pytest.mark.parametrize("Hq,Hkv,D,n,B,prefix,own", [
    (8, 1, 128, 1, 20, 3000, 100), (8, 2, 64, 4, 24, 4000, 300), (4, 4, 128, 1, 3, 2000, 40)])
def test_steps_have_two_parts(Hq, Hkv, D, n, B, prefix, own, flags):
    out, want, _, total = call(Hq, Hkv, D, n, B, prefix, own, flags)
    assert ((out - want).abs() <= (2.0 ** -16 + ROUNDING) * total).all()


@pytest.mark.parametrize("flags", [0, TC, WHOLE])
@pytest.mark.parametrize("Hq,Hkv,D,n,B,prefix,own", [(8, 2, 128, 150, 3, 3000, 200), (8, 1, 64, 40, 6, 2000, 900)])
def test_prompts_have_one(Hq, Hkv, D, n, B, prefix, own, flags):
    out, want, spread, total = call(Hq, Hkv, D, n, B, prefix, own, flags)
    err = out - want
    assert (err.abs() <= 7.6 * 2.0 ** -8 * spread + ROUNDING * total).all()
    assert err.norm() / want.norm() <= 1.02 * 2.0 ** -8 / math.sqrt(3)
