"""How far bf16 cross attention on the tensor cores is from fp64 where its outputs are small: rows
over many states, whose outputs shrink like the root of the sum of squared weights, far below
the 2e-3 that holds for every row.

Weights p_t (normalised; the sum l is of unrounded ones) go into the product with V
rounded to bf16 where none of a row's is above a twelfth, else in two parts.  So
  out_d - exact = sum_t p_t e_t v_td,   |e_t| <= 2^-8, of mean 0, and E e^2 <= 2^-16 / 3
(an error of at most half a step, uniform; the value at least 2^k where the step is 2^(k-7)).
With v drawn independently, its root mean square over all outputs is at most 2^-8 / sqrt(3) of
the outputs' own, 2.26e-3; 2 % more for the draw.  Of a single output, by Hoeffding's bound for
independent e_t: beyond 7.6 * 2^-8 S with S^2 = sum p_t^2 v_td^2 in one of 1e12.  Beside that,
products of bf16 values accumulate in fp32: at most 2^-23 of sum p |v| for each of 256 products,
2^-15, and the scores' rounding 2e-5 of the weights (as for the attention weights)."""
import math

import pytest
import torch

import exact_causal_gqa_gb300 as atlas

pytestmark = pytest.mark.gpu


def rows(Hq, Hkv, D, q, lens, dtype, seed, P=64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, width = len(lens), -(-max(lens) // P)
    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    x = normal(B, Hq, q, D), normal(B * width, Hkv, P, D), normal(B * width, Hkv, P, D)
    table = torch.randperm(B * width, generator=g, device="cuda").int().reshape(B, width)
    return (*x, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))


def exact(q, k, v, table, lens, scale):
    """Per sequence: outputs, sqrt(sum p^2 v^2) and sum p |v|, [Hq][q][D] in fp64."""
    G = q.shape[1] // k.shape[1]
    for b, L in enumerate(lens.tolist()):
        kk, vv = (x[table[b].long()].transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :L].double()
                  .repeat_interleave(G, 0) for x in (k, v))
        p = torch.softmax(q[b].double() @ kk.transpose(1, 2) * scale, -1)
        yield b, p @ vv, (p ** 2 @ vv ** 2).sqrt(), p @ vv.abs()


@pytest.mark.parametrize("Hq,Hkv,D,q,lens,flags", [
    (8, 2, 128, 300, [4000, 1500, 700], 0), (8, 2, 128, 300, [4000, 1500, 700], atlas.DEBUG_TC_DIRECT),
    (8, 8, 64, 130, [3000, 4096], 0), (6, 2, 64, 500, [2111], atlas.DEBUG_TC_DIRECT)])
def test_bf16_outputs_of_many_states(Hq, Hkv, D, q, lens, flags):
    x = rows(Hq, Hkv, D, q, lens, torch.bfloat16, D + q)
    out = atlas.cross(*x, Hq, Hkv, D, 64, D ** -0.5, out_dtype=torch.float32, debug_flags=flags)
    for b, want, spread, total in exact(*x, D ** -0.5):
        err = out[b].double() - want
        assert (err.abs() <= 7.6 * 2.0 ** -8 * spread + (2.0 ** -15 + 2e-5) * total).all()
        assert err.norm() / want.norm() <= 1.02 * 2.0 ** -8 / math.sqrt(3)
