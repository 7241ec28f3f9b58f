"""Attention over packed prompts where each running CTA takes several units one after the other
(their copies, barriers and tensor memory used again), in each of the kernel's variants, against
float64 with the tolerances of test_gpu_prompt_attention.py.  The plan query says that a shape
still gets its variant and has at least twice as many units as the device has SMs."""
import math

import pytest
import torch

from gpu_helpers import lib
from test_gpu_prompt_attention import bf16, check, run, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

SHAPES = [  # variant, query lengths, key lengths, heads, key heads, dk, dv
    ("turns", [4096], [5200], 20, 20, 192, 128),
    ("turns", [2600], [5400], 40, 20, 64, 64),
    ("turns", [3000, 0, 1300, 2000], [7000, 10, 6000, 8000], 16, 8, 128, 128),
    ("plain", [400] * 24, [400] * 24, 16, 16, 192, 128),
    ("plain", [0, 700, 1, 129, 0, 0, 333, 256] * 3, [0, 700, 5, 129, 40, 0, 900, 256] * 3, 16, 16, 64, 64),
    ("plain", [300, 17, 511] * 5, [300, 170, 512] * 5, 28, 4, 128, 80),
    ("pairs", [1] * 90, [100 + 13 * i for i in range(90)], 64, 8, 128, 128),
    ("pairs", [3, 1, 40, 5] * 12, [300, 0, 1000, 129] * 12, 16, 16, 64, 64),
]


def of_plan(m, shape):
    variant, q_lens, kv_lens, heads, kv_heads, _, dv = shape
    p = m.mla_prompt_attention_plan(sum(q_lens), sum(kv_lens), len(q_lens), heads, kv_heads, dv)
    assert p["variant"] == variant, p
    assert p["units"] >= 2 * torch.cuda.get_device_properties(0).multi_processor_count, p
    return shape[1:]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{len(s[1])}x{max(s[1])}-{max(s[2])}-{s[3]}-{s[4]}-{s[5]}-{s[6]}")
def test_units_one_after_the_other(shape, causal):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(shape[1]) + shape[5])
    q, k, v, qs, ks, scale, out, lse = run(m, g, *of_plan(m, shape), causal=causal)
    again, _ = m.mla_prompt_attention(q, k, v, qs, ks, scale, causal=causal)
    assert torch.equal(again, out)
    assert m.mla_device_fault() == 0


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], SHAPES[4], SHAPES[6]],
                         ids=lambda s: f"{s[0]}-{len(s[1])}x{max(s[1])}-{max(s[2])}-{s[3]}-{s[4]}")
def test_values_that_are_no_numbers_in_later_units(shape):
    """An infinity or NaN in one position of every sequence reaches the tokens that see it, and no others."""
    m = lib()
    q_lens, kv_lens, heads, kv_heads, dk, dv = of_plan(m, shape)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    q, k, v = bf16(g, sum(q_lens), heads, dk), bf16(g, sum(kv_lens), kv_heads, dk), bf16(g, sum(kv_lens), kv_heads, dv)
    args = (starts(q_lens), starts(kv_lens), 1 / math.sqrt(dk))
    clean, _ = m.mla_prompt_attention(q, k, v, *args)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    v2, q0, k0 = v.clone(), 0, 0
    for i, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        if nk:
            for h in range(kv_heads):  # within the last 300, so that the tokens of most units see it or not
                at, dim = nk - 1 - (37 * i + 41 * h) % min(nk, 300), (5 * i + h) % dv
                v2[k0 + at, h, dim] = (math.inf, -math.inf, math.nan)[(i + h) % 3]
                first = max(0, at - (nk - nq))
                group = heads // kv_heads
                bad[q0 + first:q0 + nq, h * group:(h + 1) * group, dim] = True
        q0, k0 = q0 + nq, k0 + nk
    out, _ = m.mla_prompt_attention(q, k, v2, *args)
    assert torch.equal(out[~bad], clean[~bad])
    assert not out[bad].isfinite().any()
    assert m.mla_device_fault() == 0


@pytest.mark.parametrize("dk,dv", [(64, 128), (32, 72), (8, 128), (128, 8), (192, 16), (192, 64)])
def test_dims_of_different_chunks(dk, dv):
    """Fewer dims of keys than of values, and the other way round."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(dk + dv)
    for causal in (True, False):
        run(m, g, [150, 1, 300], [260, 700, 300], 6, 2, dk, dv, causal=causal)
        run(m, g, [2, 1], [5000, 300], 8, 1, dk, dv, causal=causal)
