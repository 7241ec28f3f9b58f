"""Norms and rotation of queries and keys, alone and into the cache, against float64."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import lib, u16

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
INV = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)


@pytest.fixture(scope="module")
def m():
    return lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def bf16(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def turn64(x, positions, offset, interleaved, inv=None):
    """(rotated, magnitude of each value's pair) of float64 x [n, H, D]."""
    x = x.clone()
    a = positions.double()[:, None, None] * (INV if inv is None else inv).to(x.device)
    c, s = a.cos(), a.sin()
    part = x[..., offset:offset + 64]
    p, q = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :32], part[..., 32:])
    lo, hi, mag = p * c - q * s, q * c + p * s, p.abs() + q.abs()
    size = x.abs()
    if interleaved:
        x[..., offset:offset + 64] = torch.stack([lo, hi], -1).flatten(-2)
        size[..., offset:offset + 64] = torch.stack([mag, mag], -1).flatten(-2)
    else:
        x[..., offset:offset + 64] = torch.cat([lo, hi], -1)
        size[..., offset:offset + 64] = torch.cat([mag, mag], -1)
    return x, size


def heads64(x, w, positions, offset, interleaved, eps=EPS):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    return turn64(x, positions, offset, interleaved)


def assert_heads(got, ref, size):
    # one rounding to bf16 (2^-8 of the value); before it float arithmetic:
    # the sum of at most 256 squares (8 in a row, then 5 levels), rsqrt, two
    # products and the rotation, each 2^-24 of the pair's magnitude, and the
    # angle's 2^-25 of a turn: below 2^-18 of that magnitude together
    over = (got.double() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -18 * size)
    assert over.max() <= 0, over.max().item()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,hq,hk,dim,offset", [
    (1, 1, 0, 64, 0), (1, 16, 1, 128, 0), (3, 5, 2, 128, 64), (7, 16, 16, 192, 128), (33, 3, 7, 256, 192),
    (129, 32, 1, 128, 8), (2, 1, 1, 72, 8), (5, 2, 3, 200, 40), (1000, 16, 4, 192, 128),
])
def test_heads(m, n, hq, hk, dim, offset, interleaved):
    g = gen(n + dim)
    q, k = bf16(g, n, hq, dim, scale=3.0), bf16(g, n, max(hk, 1), dim, scale=0.1)
    wq, wk = bf16(g, dim), bf16(g, dim)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32)
    qo, ko = m.mla_qk_norm_rope(q, k if hk else None, pos, INV.to(DEV), wq, wk, EPS, offset, interleaved)
    torch.cuda.synchronize()
    assert_heads(qo, *heads64(q, wq, pos, offset, interleaved))
    if hk:
        assert_heads(ko, *heads64(k, wk, pos, offset, interleaved))
    else:
        assert ko is None


def test_without_weights_only_rotates(m):
    g = gen(1)
    q = bf16(g, 20, 4, 128)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    qo, _ = m.mla_qk_norm_rope(q, None, pos, INV.to(DEV), rope_offset=32)
    torch.cuda.synchronize()
    assert torch.equal(qo[..., :32], q[..., :32]) and torch.equal(qo[..., 96:], q[..., 96:])
    assert torch.equal(qo[0], q[0])  # position 0 turns nothing
    assert_heads(qo, *heads64(q, None, pos, 32, True))


@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 24 + 1, -3])
def test_far_positions(m, far):
    """Angles of positions that a float product would lose; a negative one turns backwards."""
    g = gen(2)
    q = bf16(g, 4, 2, 64)
    pos = torch.tensor([far, far - 1, far // 3, 0], dtype=torch.int32, device=DEV)
    # frequencies that are whole multiples of 2^-20: position x frequency is exact in float64
    inv = torch.round(INV * 2 ** 20) / 2 ** 20
    qo, _ = m.mla_qk_norm_rope(q, None, pos, inv.to(DEV))
    torch.cuda.synchronize()
    # inv_freq / 2 pi is a float64, so a far position's angle is known to position x inv_freq x 2^-52
    ref, size = turn64(q.double(), pos, 0, True, inv)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -18 + abs(far) * 2.0 ** -51) * size
    assert ((qo.double() - ref).abs() <= tol).all()


def test_strides_and_in_place(m):
    """Queries and keys as slices of one projection, rotated in place; head-major outputs."""
    g = gen(3)
    n, hq, hk, dim = 37, 6, 2, 128
    both = bf16(g, n, hq + hk, dim)
    start = both.clone()
    w = bf16(g, dim)
    pos = torch.randint(0, 5000, (n,), generator=g, device=DEV, dtype=torch.int32)
    q, k = both[:, :hq], both[:, hq:]
    major = torch.full((hk, n, dim), float("nan"), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    m.mla_qk_norm_rope(q, k, pos, INV.to(DEV), w, w, EPS, 0, False, q_out=q, k_out=major)
    torch.cuda.synchronize()
    assert_heads(both[:, :hq], *heads64(start[:, :hq], w, pos, 0, False))
    assert_heads(major, *heads64(start[:, hq:], w, pos, 0, False))
    assert torch.equal(both[:, hq:], start[:, hq:])
    wide = bf16(g, n, 3, 192)  # only the last 64 values of each head
    part = wide[..., 128:]
    keep = wide[..., :128].clone()
    before = part.clone()
    m.mla_qk_norm_rope(part, None, pos, INV.to(DEV), q_out=part)
    torch.cuda.synchronize()
    assert torch.equal(wide[..., :128], keep)
    assert_heads(part, *heads64(before, None, pos, 0, True))


def test_zero_and_infinite_heads(m):
    """A head of zeros stays zeros; a NaN or infinity stays in its head."""
    g = gen(4)
    q = bf16(g, 3, 4, 128)
    clean = q.clone()
    q[0, 1] = 0
    q[1, 2, 70] = float("nan")
    q[2, 3, 5] = float("inf")
    w = bf16(g, 128)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    qo, _ = m.mla_qk_norm_rope(q, None, pos, INV.to(DEV), w)
    co, _ = m.mla_qk_norm_rope(clean, None, pos, INV.to(DEV), w)
    torch.cuda.synchronize()
    assert (qo[0, 1] == 0).all() and torch.isnan(qo[1, 2]).all()
    same = torch.ones((3, 4), dtype=torch.bool, device=DEV)
    same[0, 1] = same[1, 2] = same[2, 3] = False
    assert torch.equal(qo[same], co[same])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,hq", [(1, 0), (9, 16), (300, 3)])
def test_append(m, fmt, interleaved, n, hq):
    g = gen(5 + n)
    rb = (352, 576)[fmt]
    kv = bf16(g, n, 576 + 24, scale=4.0)[:, :576]  # rows 600 apart
    w = bf16(g, 512)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32)
    nb = -(-n // 64) + 2
    stride = 64 * rb + 32
    slots = torch.randperm(nb * 64, generator=g, device=DEV)[:n].contiguous()
    if n > 5:
        slots[3], slots[5] = -1, nb * 64  # skipped
    pool = torch.full((nb, stride), 0xAB, dtype=torch.uint8, device=DEV)
    q = bf16(g, n, hq, 192) if hq else None
    wq = bf16(g, 192)
    qo = m.mla_kv_norm_rope_append(kv, w, pos, INV.to(DEV), slots, pool, nb, 64, stride, fmt, EPS, interleaved, q, wq,
                                   128)
    torch.cuda.synchronize()
    if hq:
        assert_heads(qo, *heads64(q, wq, pos, 128, interleaved))
    else:
        assert qo is None
    # The bytes that the oracle writes for the bf16 rows.  Float arithmetic may
    # round a value that lies within 2^-18 of two bf16 values' middle either way:
    # where the rows of values 2^-18 lower and higher differ, either may stand.
    lat = kv[:, :512].double()
    lat = lat / torch.sqrt(lat.square().mean(-1, keepdim=True) + EPS) * w.double()
    rope, size = turn64(kv[:, None, 512:].double(), pos, 0, interleaved)
    rope, size = rope[:, 0], size[:, 0]
    want = []
    for sign in (-1, 1):
        p = np.full((nb, stride), 0xAB, np.uint8)
        O.kv_quantize_append(u16((lat * (1 + sign * 2.0 ** -18)).to(torch.bfloat16)),
                             u16((rope + sign * 2.0 ** -18 * size).to(torch.bfloat16)), slots.cpu().numpy(),
                             p.reshape(-1), nb, 64, stride, fmt)
        want.append(p)
    got = pool.cpu().numpy()
    sure = want[0] == want[1]
    assert sure.mean() > 0.99
    assert np.array_equal(got[sure], want[0][sure])


def test_append_zero_row_and_no_tokens(m):
    pool = torch.full((1, 64, 352), 0x55, dtype=torch.uint8, device=DEV)
    kv = torch.zeros((1, 576), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    one = torch.tensor([5], dtype=torch.int32, device=DEV)
    m.mla_kv_norm_rope_append(kv, w, one, INV.to(DEV), one.long(), pool, 1, 64, 64 * 352)
    m.mla_kv_norm_rope_append(kv[:0], w, one[:0], INV.to(DEV), one[:0].long(), pool, 1, 64, 64 * 352)
    torch.cuda.synchronize()
    # zero times a negative cosine is -0: the rope bytes may carry a sign, nothing else
    assert (pool[0, 5, :288] == 0).all() and ((pool[0, 5, 288:] & 0x7F) == 0).all()
    assert (pool[0, :5] == 0x55).all() and (pool[0, 6:] == 0x55).all()


def test_refusals(m):
    g = gen(6)
    q = bf16(g, 4, 2, 128)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    inv = INV.to(DEV)
    w = bf16(g, 128)
    for kw, error in ((dict(rope_offset=65), m.MlaError), (dict(rope_offset=4), m.MlaError),
                      (dict(rope_offset=-8), m.MlaError), (dict(eps=0.0), m.MlaError),
                      (dict(q_weight=w[:64]), ValueError), (dict(q_weight=w.float()), TypeError),
                      (dict(q_out=q[:2]), ValueError)):
        with pytest.raises(error):
            m.mla_qk_norm_rope(q, None, pos, inv, **kw)
    with pytest.raises(m.MlaError):  # one row of the output would be all rows
        m.mla_qk_norm_rope(q, None, pos, inv, q_out=q[:1].expand(4, 2, 128))
    with pytest.raises(m.MlaError) as e:
        m.mla_qk_norm_rope(bf16(g, 4, 2, 264), None, pos, inv)
    assert e.value.status == 2
    with pytest.raises(m.MlaError):
        m.mla_qk_norm_rope(bf16(g, 4, 2, 132)[..., 2:130], None, pos, inv)  # heads not 16-byte aligned
    with pytest.raises(ValueError):
        m.mla_qk_norm_rope(q, None, pos[:3], inv)
    with pytest.raises(TypeError):
        m.mla_qk_norm_rope(q, None, pos, inv.float())
    with pytest.raises(TypeError):
        m.mla_qk_norm_rope(q.float(), None, pos, inv)
    pool = torch.zeros((1, 64, 352), dtype=torch.uint8, device=DEV)
    kv, lw = bf16(g, 4, 576), bf16(g, 512)
    with pytest.raises(ValueError):
        m.mla_kv_norm_rope_append(kv, lw, pos, inv, pos.long(), pool, 2, 64, 64 * 352)
    with pytest.raises(m.MlaError):
        m.mla_kv_norm_rope_append(kv, lw, pos, inv, pos.long(), pool, 1, 64, 64 * 352 - 16)
    with pytest.raises(ValueError):
        m.mla_kv_norm_rope_append(kv[:, :512], lw, pos, inv, pos.long(), pool, 1, 64, 64 * 352)
    e = q[:0]
    out, _ = m.mla_qk_norm_rope(e, None, pos[:0], inv)
    assert out.shape == (0, 2, 128)
