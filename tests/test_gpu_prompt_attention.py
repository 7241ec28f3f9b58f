"""Attention over packed prompts against float64.

Tolerances.  With p the exact softmax, A = sum p |v| and Z = the largest
scale sum |q k| of the call:
  scores    a float32 product of D values in the tensor core (D / 16 steps, each
            within 2^-22 of the magnitudes so far), its product with the scale and
            the difference to the reference (2^-24 of the larger): within
            dz = (D / 16 x 2^-22 + 4 x 2^-24) Z, and ex2 within 2^-22
  sum       n keys in four partial sums, one rounding each: n / 4 x 2^-24, and of a
            few joined
  out       a weight rounded to bf16 2^-8 of itself, out to bf16 2^-8 of itself:
            2^-8 A + 2^-8 |out| + 2 (dz + 2^-22 + (n / 4 + 16) x 2^-24) A, the
            product's own sum n / 16 x 2^-22 A
  lse       dz + 2^-22 + (n / 4 + 16) x 2^-24, and 4 roundings of its own size"""
import math

import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bf16(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def starts(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def reference(q, k, v, qs, ks, scale, causal):
    """(out, lse, A, Z) in float64 of every token in a sequence; NaN elsewhere."""
    total, heads, _ = q.shape
    out = torch.full((total, heads, v.shape[2]), math.nan, dtype=torch.float64, device=DEV)
    mag, lse = out.clone(), torch.full((total, heads), math.nan, dtype=torch.float64, device=DEV)
    top = 0.0
    group = heads // k.shape[1]
    for b in range(len(qs) - 1):
        q0, q1, k0, k1 = qs[b], qs[b + 1], ks[b], ks[b + 1]
        nq, nk = q1 - q0, k1 - k0
        if nq == 0:
            continue
        seen = torch.ones((nq, nk), dtype=torch.bool, device=DEV)
        if causal:
            seen = seen.tril(nk - nq)
        for h in range(heads):
            x, y, w = q[q0:q1, h].double(), k[k0:k1, h // group].double(), v[k0:k1, h // group].double()
            z = (x @ y.t() * scale).masked_fill(~seen, -math.inf)
            if nk:
                top = max(top, abs(scale) * (x.abs() @ y.abs().t()).max().item())
            lse[q0:q1, h] = torch.logsumexp(z, -1) if nk else -math.inf
            p = torch.softmax(z, -1).masked_fill(~seen.any(-1, keepdim=True), 0.0)
            out[q0:q1, h], mag[q0:q1, h] = p @ w, p @ w.abs()
    return out, lse, mag, top


def check(out, lse, q, k, v, qs, ks, scale, causal):
    want, want_lse, mag, top = reference(q, k, v, qs, ks, scale, causal)
    n = max([b - a for a, b in zip(ks, ks[1:])] + [1])
    dz = (q.shape[2] / 16 * 2.0 ** -22 + 4 * 2.0 ** -24) * top
    more = dz + 2.0 ** -22 + (n / 4 + 16) * 2.0 ** -24
    ours = ~want_lse.isnan()
    err = (out.double() - want).abs()[ours]
    tol = (2.0 ** -8 + 2 * more + n / 16 * 2.0 ** -22) * mag[ours] + 2.0 ** -8 * want.abs()[ours]
    assert (err <= tol).all(), (err - tol).max().item()
    if lse is not None:
        a, b = lse.double()[ours], want_lse[ours]
        assert torch.equal(a.isneginf(), b.isneginf())
        fin = b.isfinite()
        assert ((a - b).abs()[fin] <= more + 4 * 2.0 ** -24 * (b.abs()[fin] + 1)).all(), (a - b).abs()[fin].max().item()


def run(m, g, q_lens, kv_lens, heads, kv_heads, dk, dv, causal=True, scale=None, q_scale=1.0):
    qs, ks = starts(q_lens), starts(kv_lens)
    q, kv = bf16(g, sum(q_lens), heads, dk, scale=q_scale), bf16(g, sum(kv_lens), kv_heads, dk + dv)
    k, v = kv[..., :dk], kv[..., dk:]
    scale = 2.0 / math.sqrt(dk) if scale is None else scale
    lse = torch.full((sum(q_lens), heads), 7.0, device=DEV)
    out, _ = m.mla_prompt_attention(q, k, v, qs, ks, scale, causal=causal, lse=lse)
    check(out, lse, q, k, v, qs.tolist(), ks.tolist(), scale, causal)
    return q, k, v, qs, ks, scale, out, lse


SHAPES = [  # query lengths, key lengths, heads, key heads, dk, dv
    ([1], [1], 1, 1, 64, 64),
    ([1, 1, 1], [1, 2, 129], 8, 8, 64, 64),
    ([127, 128, 129], [127, 128, 129], 2, 2, 64, 64),
    ([17, 3, 11], [17, 3, 11], 8, 8, 64, 64),
    ([300], [300], 3, 3, 192, 128),
    ([257, 1, 500], [257, 1, 500], 4, 2, 192, 128),
    ([130, 64], [1000, 64], 16, 16, 192, 128),
    ([200, 10], [333, 1024], 28, 4, 128, 128),
    ([1] * 9, [1, 64, 127, 128, 129, 255, 256, 257, 3000], 64, 8, 128, 128),
    ([5, 4, 3], [700, 4, 90], 15, 3, 96, 80),
    ([3, 2], [100, 200], 128, 1, 128, 128),
    ([2], [50], 100, 1, 64, 64),
    ([100, 300], [100, 300], 6, 2, 8, 8),
    ([65], [191], 2, 1, 72, 16),
    ([40], [700], 5, 1, 136, 24),
    ([2000], [2000], 2, 2, 128, 128),
    ([700], [5000], 1, 1, 192, 128),
    ([1], [40000], 2, 1, 192, 128),
    ([300], [5200], 2, 2, 64, 64),
    ([600, 300, 40], [9000, 7000, 40], 4, 1, 128, 128),
    ([700], [5300], 1, 1, 192, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(s[0])}-{max(s[1])}-{s[2]}-{s[3]}-{s[4]}-{s[5]}")
def test_sizes(shape, causal):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(shape[0]) + shape[4])
    run(m, g, *shape, causal=causal)


def test_empty_sequences_and_tokens_that_see_nothing():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for causal in (True, False):
        *_, out, lse = run(m, g, [0, 3, 200, 0, 5, 140], [4, 0, 150, 0, 3, 20], 4, 2, 128, 128, causal)
        assert (out[:3] == 0).all() and lse[:3].isneginf().all()
        if causal:
            assert (out[3:53] == 0).all() and lse[3:53].isneginf().all() and lse[53:203].isfinite().all()
    # no keys at all
    q, qs = bf16(g, 5, 2, 64), starts([5])
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    lse = torch.ones((5, 2), device=DEV)
    out, _ = m.mla_prompt_attention(q, none, none, qs, starts([0]), 0.1, lse=lse)
    assert (out == 0).all() and lse.isneginf().all()
    assert m.mla_prompt_attention(q[:0], none, none, starts([0]), starts([0]), 0.1)[0].shape == (0, 2, 64)
    assert m.mla_prompt_attention(q, q, q, starts([]), starts([]), 0.1, out=torch.ones_like(q))[0].eq(1).all()


def test_tokens_outside_the_sequences_stay():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    q, k, v = bf16(g, 60, 4, 64), bf16(g, 3000, 4, 64), bf16(g, 3000, 4, 64)
    for ends in ([11, 12, 40], [11, 12, 12]):  # rows behind the last sequence; with splits and without
        for kv in ([7, 30, 40], [7, 1500, 2990]):
            qs, ks = torch.tensor(ends, dtype=torch.int32, device=DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
            out, lse = torch.full((60, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((60, 4), 5.0, device=DEV)
            m.mla_prompt_attention(q, k, v, qs, ks, 0.2, out=out, lse=lse)
            check(out, lse, q, k, v, ends, kv, 0.2, True)
            rest = [t for t in range(60) if not ends[0] <= t < ends[-1]]
            assert (out[rest] == 3).all() and (lse[rest] == 5).all()


def test_starts_outside_the_tensors_are_cut():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    q, k, v = bf16(g, 50, 2, 64), bf16(g, 80, 2, 64), bf16(g, 80, 2, 64)
    wild_q = torch.tensor([-5, 20, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    wild_k = torch.tensor([-2 ** 31, 30, 1000], dtype=torch.int32, device=DEV)
    out, _ = m.mla_prompt_attention(q, k, v, wild_q, wild_k, 0.2)
    want, _ = m.mla_prompt_attention(q, k, v, starts([20, 30]), starts([30, 50]), 0.2)
    assert torch.equal(out, want)
    # decreasing starts: any values, but nothing outside the tensors is touched
    m.mla_prompt_attention(q, k, v, torch.tensor([30, 10, 50], dtype=torch.int32, device=DEV),
                           torch.tensor([80, 0, 40], dtype=torch.int32, device=DEV), 0.2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale,q_scale", [(-0.2, 1.0), (0.0, 1.0), (0.125, 40.0), (1e-3, 1.0)])
def test_scales(scale, q_scale):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    run(m, g, [200, 33], [300, 33], 4, 2, 128, 128, True, scale, q_scale)


def test_late_maxima():
    """The largest scores come last, in steps below and above the maximum's lag, before a flat tail."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    q, k, v = bf16(g, 256, 1, 64), bf16(g, 1024, 1, 64, scale=0.05), bf16(g, 1024, 1, 64)
    q[:, 0, 0] = 8.0
    for step in (0.4, 3.0, 30.0, -30.0):
        k[:, 0, 0] = (torch.arange(1024, device=DEV) // 64 * step).to(torch.bfloat16)
        lse = torch.empty((256, 1), device=DEV)
        out, _ = m.mla_prompt_attention(q, k, v, starts([256]), starts([1024]), 1.0, lse=lse)
        check(out, lse, q, k, v, [0, 256], [0, 1024], 1.0, True)


def test_values_that_are_no_numbers_stay_where_they_are_seen():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    q_lens, kv_lens = [300, 70, 5], [450, 70, 600]
    for dk, dv in ((64, 64), (192, 128)):
        for causal in (True, False):
            qs, ks = starts(q_lens), starts(kv_lens)
            q, k, v = bf16(g, 375, 2, dk), bf16(g, 1120, 2, dk), bf16(g, 1120, 2, dv)
            args = (qs, ks, 0.2)
            clean_lse = torch.empty((375, 2), device=DEV)
            clean, _ = m.mla_prompt_attention(q, k, v, *args, causal=causal, lse=clean_lse)
            v2, k2, q2 = v.clone(), k.clone(), q.clone()
            v2[200, 0, 3] = math.nan      # sequence 0, position 200: seen from query 50 on
            v2[449, 0, 5] = math.inf      # its last position
            v2[300, 1, 7] = -math.inf
            v2[450, 1, 9] = math.nan      # sequence 1's first
            k2[460, 0, 1] = math.nan      # sequence 1, position 10, as a key
            k2[1119, 1, 2] = math.inf     # the last key of all
            q2[372, 0, 0] = math.nan      # one query
            lse = torch.empty((375, 2), device=DEV)
            out, _ = m.mla_prompt_attention(q2, k2, v2, *args, causal=causal, lse=lse)
            bad, bad_lse = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(lse, dtype=torch.bool)
            bad[50 if causal else 0:300, 0, 3] = True
            bad[299 if causal else 0:300, 0, 5] = True
            bad[150 if causal else 0:300, 1, 7] = True
            bad[300:370, 1, 9] = True
            bad[310 if causal else 300:370, 0] = True
            bad_lse[310 if causal else 300:370, 0] = True
            bad[374 if causal else 370:375, 1] = True
            bad_lse[374 if causal else 370:375, 1] = True
            bad[372, 0], bad_lse[372, 0] = True, True
            assert torch.equal(~out.isfinite() & ~bad, torch.zeros_like(bad))
            assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad_lse], clean_lse[~bad_lse])
            assert out[50 if causal else 0:300, 0, 3].isnan().all() and out[300:370, 1, 9].isnan().all()
            assert out[299, 0, 5] == math.inf and (out[150:300, 1, 7] == -math.inf).all()
            assert lse[310:370, 0].isnan().all() and lse[372, 0].isnan()


def test_strides():
    """Heads before tokens, slices of wider heads, one key head shared by stride, out in a larger buffer."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    qs, ks = starts([150]), starts([260])
    q = bf16(g, 6, 150, 200).transpose(0, 1)[..., 8:200]
    k, v = bf16(g, 260, 2, 192), bf16(g, 2, 260, 128).transpose(0, 1)
    room = torch.full((150, 6, 160), 2.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((150, 6), device=DEV)
    out, _ = m.mla_prompt_attention(q, k, v, qs, ks, 0.1, out=room[..., 16:144], lse=lse)
    check(out, lse, q, k, v, [0, 150], [0, 260], 0.1, True)
    assert (room[..., :16] == 2).all() and (room[..., 144:] == 2).all()
    want, _ = m.mla_prompt_attention(q.contiguous(), k, v.contiguous(), qs, ks, 0.1)
    assert torch.equal(out, want)


def test_streams_capture_and_new_inputs():
    """Another stream; a captured call replayed over new lengths and values; two captured calls on one workspace."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    q, k, v = bf16(g, 12, 8, 128), bf16(g, 9000, 2, 128), bf16(g, 9000, 2, 128)
    qs, ks = starts([4, 4, 4]), starts([3000, 2500, 3500])
    need = m.mla_prompt_attention_workspace_size(12, 9000, 3, 8, 2, 128)
    assert need > 0
    want, _ = m.mla_prompt_attention(q, k, v, qs, ks, 0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = m.mla_prompt_attention(q, k, v, qs, ks, 0.2, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(want) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o in outs:
            m.mla_prompt_attention(q, k, v, qs, ks, 0.2, out=o, workspace=ws)
    q.copy_(bf16(g, 12, 8, 128))
    qs.copy_(starts([1, 9, 2]))
    ks.copy_(starts([10, 8000, 990]))
    graph.replay()
    torch.cuda.synchronize()
    check(outs[0], None, q, k, v, qs.tolist(), ks.tolist(), 0.2, True)
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(outs[0], m.mla_prompt_attention(q, k, v, qs, ks, 0.2)[0])


def test_refusals():
    m = lib()
    q, k, v = (torch.zeros((10, 4, 64), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    s = starts([10])
    call = m.mla_prompt_attention
    for bad in (lambda: call(q, k[:5], v, s, s, 1.0), lambda: call(q, k[..., :32], v, s, s, 1.0),
                lambda: call(q, k, v, s, s[:1], 1.0), lambda: call(q.cpu(), k, v, s, s, 1.0),
                lambda: call(q, k, v, s, s, 1.0, out=q[:5]), lambda: call(q[..., ::2], k[..., ::2], v, s, s, 1.0),
                lambda: call(q, k, v, s, s, 1.0, lse=torch.zeros((10, 3), device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        call(q.float(), k, v, s, s, 1.0)
    with pytest.raises(TypeError):
        call(q, k, v, s.long(), s, 1.0)
    for bad in (lambda: call(q[:, :3], k[:, :2], v[:, :2], s, s, 1.0), lambda: call(q, k, v, s, s, math.nan),
                lambda: call(q[..., :60], k[..., :60], v, s, s, 1.0), lambda: call(q, k, v[..., :4], s, s, 1.0),
                lambda: call(q, k, v, s, s, 1.0, out=torch.empty(10 * 4 * 64, dtype=torch.bfloat16, device=DEV).as_strided(
                    (10, 4, 64), (64, 64, 1)))):
        with pytest.raises(m.MlaError):
            bad()


def test_no_keys_whatever_their_strides():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    q = bf16(g, 5, 4, 64)
    k = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=DEV).expand(0, 2, 64)
    lse = torch.zeros((5, 4), device=DEV)
    out, _ = m.mla_prompt_attention(q, k, k, starts([2, 3]), starts([0, 0]), 0.1, lse=lse)
    assert (out == 0).all() and lse.isneginf().all()


def test_a_repeated_key_head_is_refused():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    q, k = bf16(g, 7, 4, 64), bf16(g, 7, 1, 64)
    with pytest.raises(m.MlaError):
        m.mla_prompt_attention(q, k.expand(7, 4, 64), k.expand(7, 4, 64), starts([7]), starts([7]), 0.1)
    out, _ = m.mla_prompt_attention(q, k, k, starts([7]), starts([7]), 0.1)  # one key head for all
    check(out, None, q, k, k, [0, 7], [0, 7], 0.1, True)


@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_the_largest_scales(scale):
    """Scores 0 and of the order of the scale: all weight lies on the largest."""
    m = lib()
    q = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device=DEV)
    k[1, 0, 0] = -2.0 ** -10 if scale > 0 else 2.0 ** -10
    v = torch.tensor([1.0, 100.0, 3.0], device=DEV)[:, None, None].expand(3, 1, 64).to(torch.bfloat16).contiguous()
    out, _ = m.mla_prompt_attention(q, k, v, starts([1]), starts([3]), scale)
    assert (out == 2.0).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", [
    ([300, 1, 1, 1], [500, 3000, 700, 129], 2, 2, 128, 128),
    ([1, 140, 2], [4000, 4100, 257], 1, 1, 192, 128),
    ([2, 3, 1, 0, 4], [257, 128, 129, 500, 0], 8, 2, 64, 64),
    ([9, 7], [1290, 3], 12, 1, 96, 80),
    ([128, 128], [1000, 385], 1, 1, 64, 64),
])
def test_few_rows_over_many_keys(shape, causal):
    """One tile of rows for most sequences, whose tiles of keys two groups share; others with
    more rows, one tile of keys or none in the same call."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    q, k, v, qs, ks, scale, out, lse = run(m, g, *shape, causal=causal)
    again, _ = m.mla_prompt_attention(q, k, v, qs, ks, scale, causal=causal)
    assert torch.equal(again, out)
    # scores that grow along the keys, and ones that fall: either half has the largest
    for sign in (1, -1):
        k2 = (k.float() * 0.1 + sign * torch.linspace(-1, 1, k.shape[0], device=DEV)[:, None, None]).to(torch.bfloat16)
        q2 = (q.float() * 0.1 + 1).to(torch.bfloat16)
        lse = torch.empty_like(lse)
        out, _ = m.mla_prompt_attention(q2, k2, v, qs, ks, 0.7, causal=causal, lse=lse)
        check(out, lse, q2, k2, v, qs.tolist(), ks.tolist(), 0.7, causal)
