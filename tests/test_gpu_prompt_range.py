"""Attention over packed prompts whose scores are large, up to the end of float32's range
and past it.

Scores here are whole numbers times a power of two, so that float32 holds them
exactly, and far enough apart that a weight is 0 or that of the largest: the
expected row is a mean of values.  Tolerances: the weights of a row are one number (a
power of two of what the rounding of the largest's product leaves), which bf16
rounds by 2^-8 of itself and so out by that; the product's sum of n values n / 16 x
2^-22 of their magnitudes and the division 2^-22, bf16 out 2^-8 of itself; lse a
logarithm (2^-22 of up to 16) and 4 roundings."""
import math

import pytest
import torch

from gpu_helpers import lib
from test_gpu_prompt_attention import bf16, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# query lengths, key lengths, heads, key heads, dims: one slice, both tiles of a CTA on the
# same rows, slices joined, many units
SHAPES = [([3], [3], 1, 1, 64), ([200, 40], [300, 500], 4, 2, 128), ([128], [700], 1, 1, 64),
          ([1, 2], [40000, 900], 2, 1, 128), ([5], [9000], 8, 2, 64), ([700], [5000], 1, 1, 128),
          ([260] * 20, [300] * 20, 16, 16, 64)]


def expected(level, v, nq, nk, causal):
    """(out, largest level seen, its keys, magnitudes) of one sequence and head."""
    i, j = torch.arange(nq, device=DEV)[:, None], torch.arange(nk, device=DEV)
    seen = (j <= nk - nq + i) if causal else (j >= 0).expand(nq, nk)
    top = torch.where(seen, level, -100).amax(1)
    of = (seen & (level == top[:, None])).double()
    count = of.sum(1)
    n = count.clamp(min=1)[:, None]
    return of @ v.double() / n, top.double(), count, of @ v.double().abs() / n


@pytest.mark.parametrize("power", [130, 125, 100, 33, 26, 25, 21])
@pytest.mark.parametrize("levels", [(0, 9), (-8, 0), (-3, 4)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{max(s[1])}-{s[2]}-{s[3]}-{s[4]}")
def test_large_scores(shape, levels, power):
    """q.k times the scale is a small whole number x 2^power: NaN where the largest one seen is
    2^30 (base 2) or more in magnitude, however far past float32, and right for all others.
    A key in 50 has the level 0 besides."""
    m = lib()
    q_lens, kv_lens, heads, kv_heads, d = shape
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(kv_lens))
    n_q, n_k = sum(q_lens), sum(kv_lens)
    for sign, causal in ((1, True), (-1, True), (1, False)):
        level = torch.randint(*levels, (n_k, kv_heads), generator=g, device=DEV)
        level[torch.rand((n_k, kv_heads), generator=g, device=DEV) < 0.02] = 0
        q, k = torch.zeros((n_q, heads, d), device=DEV), torch.zeros((n_k, kv_heads, d), device=DEV)
        q[..., 0], k[..., 0] = 2.0 ** 30, level * sign * 2.0 ** 30
        q, k, v = q.to(torch.bfloat16), k.to(torch.bfloat16), bf16(g, n_k, kv_heads, d)
        lse = torch.full((n_q, heads), 7.0, device=DEV)
        out, _ = m.mla_prompt_attention(q, k, v, starts(q_lens), starts(kv_lens), sign * 2.0 ** (power - 60),
                                        causal=causal, lse=lse)
        q0 = k0 = 0
        for nq, nk in zip(q_lens, kv_lens):
            for h in range(heads):
                at = h * kv_heads // heads
                want, top, count, mag = expected(level[k0:k0 + nk, at], v[k0:k0 + nk, at], nq, nk, causal)
                got, got_lse = out[q0:q0 + nq, h].double(), lse[q0:q0 + nq, h].double()
                large = (top * 2.0 ** power / math.log(2.0)).abs() >= 2.0 ** 30
                assert torch.equal(got.isnan(), large[:, None].expand_as(got)) and torch.equal(got_lse.isnan(), large)
                ours = ~large
                tol = 2 * 2.0 ** -8 * want.abs() + (nk / 16 + 1) * 2.0 ** -22 * mag
                assert ((got - want).abs() <= tol)[ours].all()
                want_lse = top * 2.0 ** power + torch.log(count)
                assert ((got_lse - want_lse).abs() <= 2.0 ** -18 + 4 * 2.0 ** -24 * want_lse.abs())[ours].all()
            q0, k0 = q0 + nq, k0 + nk


@pytest.mark.parametrize("nk", [3, 300, 20000])
def test_scores_of_minus_infinity(nk):
    """Keys whose score is -infinity have no weight beside others; among themselves they have none that
    is a number."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(nk)
    q, k, v = torch.zeros((2, 1, 64), device=DEV), torch.zeros((nk, 1, 64), device=DEV), bf16(g, nk, 1, 64)
    q[..., 0] = 1
    k[:-1, 0, 0] = -math.inf  # the last is seen by the second token alone
    lse = torch.zeros((2, 1), device=DEV)
    out, _ = m.mla_prompt_attention(q.to(torch.bfloat16), k.to(torch.bfloat16), v, starts([2]), starts([nk]), 0.5, lse=lse)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert torch.equal(out[1], v[-1]) and lse[1].abs().item() <= 2.0 ** -22


@pytest.mark.parametrize("nq,heads,nk", [(1, 1, 129), (1, 1, 4000), (1, 1, 30000), (128, 160, 300), (300, 90, 129),
                                         (300, 90, 256), (300, 90, 700), (600, 40, 6000)])
@pytest.mark.parametrize("step", [1, 7, 8, 9])
def test_values_near_the_largest_float(nq, heads, nk, step):
    """The last key's score is `step` (base 2) above the ones before it, its values are 2^127: weighted
    sums with weights up to 1 stay floats.  out = 2^127 / (1 + (nk - 1) 2^-step) up to the
    tolerances above, the weights' rounding to bf16 (2^-8) and twice what the sum is off by: the
    scores' product with the scale and difference to the reference 4 x 2^-24 of up to 2^5, ex2
    2^-22, the sums of nk weights (nk / 4 + 16) x 2^-24."""
    m = lib()
    q, k = torch.zeros((nq, heads, 64), device=DEV), torch.zeros((nk, heads, 64), device=DEV)
    v = torch.zeros((nk, heads, 64), device=DEV)
    q[..., 0], k[-1, :, 0], v[-1] = 1, step, 2.0 ** 127
    v[:, :, 1] = 2.0 ** -120  # and a value that all have, near the other end
    out, _ = m.mla_prompt_attention(q.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16), starts([nq]),
                                    starts([nk]), math.log(2.0), causal=False)
    want = 2.0 ** 127 / (1 + (nk - 1) * 2.0 ** -step)
    tol = 2 * 2.0 ** -8 + nk / 16 * 2.0 ** -22 + 2 * (2.0 ** -17 + 2.0 ** -22 + (nk / 4 + 16) * 2.0 ** -24)
    got = out.double()
    rest = torch.cat([got[..., :1], got[..., 2:]], -1)
    assert ((rest / want - 1).abs() <= tol).all(), (rest / want - 1).abs().max().item()
    assert ((got[..., 1] * 2.0 ** 120 - 1).abs() <= tol).all(), got[..., 1].max().item() * 2.0 ** 120
