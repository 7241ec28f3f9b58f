"""Strides of the head sets that norm + rotation takes: outputs whose heads share
elements are refused, on the host, and no others.  Refused calls never
dereference their pointers."""
import ctypes as C

import pytest
import torch

INVALID = 1
FAKE = C.c_void_p(0x10000)


@pytest.fixture(scope="module")
def m():
    from sparse_mla_decode_kv_gb300 import build
    build.build()
    import sparse_mla_decode_kv_gb300 as m
    m.load()
    return m


def status(m, n, heads, token, head, dim=64, in_place=False):
    """Status of mla_qk_norm_rope on an output with these strides."""
    h = m._Heads(0x10000, 0x10000 if in_place else 0x20000, heads, token if in_place else 8, head if in_place else 8,
                 token, head, 0x30000)
    return m.load().mla_qk_norm_rope(C.byref(h), None, n, dim, 0, 1, 1e-6, FAKE, FAKE, None)


def overlapping(n, heads, token, head, dim):
    at = sorted(i * token + j * head for i in range(n) for j in range(heads))
    return any(b - a < dim for a, b in zip(at, at[1:]))


CASES = [(2, 2, 64, 64), (5, 2, 64, 64), (2, 2, 128, 64), (2, 2, 64, 128), (3, 3, 128, 192), (2, 3, 320, 128),
         (3, 2, 320, 128), (4, 4, 200, 72), (3, 7, 448, 64), (3, 8, 448, 64), (6, 3, 64, 384), (7, 3, 64, 384),
         (9, 5, 136, 200), (2, 9, 136, 1088), (33, 4, 64, 2112), (34, 4, 64, 2112), (5, 5, 448, 320)]
SHARED = [c for c in CASES if overlapping(*c, 64)]
APART = [c for c in CASES if not overlapping(*c, 64)]


@pytest.mark.parametrize("n,heads,token,head", SHARED)
@pytest.mark.parametrize("in_place", [False, True])
def test_overlapping_outputs_are_refused(m, n, heads, token, head, in_place):
    assert status(m, n, heads, token, head, in_place=in_place) == INVALID


@pytest.mark.parametrize("n,heads,token,head", [(2, 2, 1 << 62, 1 << 62), (1 << 40, 3, 64, 64), (3, 1 << 30, 64, 64)])
def test_strides_past_64_bits(m, n, heads, token, head):
    """Products that 64 bits do not hold; equal strides share rows whatever their size."""
    assert status(m, n, heads, token, head) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("n,heads,token,head", APART)
def test_other_strides_are_taken(m, n, heads, token, head):
    """Nested either way, or interleaved: what lies between the heads stays as it is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n * heads)
    x = torch.randn((n, heads, 64), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    inv = torch.full((32,), 0.5, dtype=torch.float64, device="cuda")
    want, _ = m.mla_qk_norm_rope(x, None, pos, inv)
    buf = torch.full(((n - 1) * token + (heads - 1) * head + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mla_qk_norm_rope(x, None, pos, inv, q_out=buf.as_strided((n, heads, 64), (token, head, 1)))
    torch.cuda.synchronize()
    expect = torch.full_like(buf, 7.0)
    expect.as_strided((n, heads, 64), (token, head, 1)).copy_(want)
    assert torch.equal(buf, expect)


@pytest.mark.gpu
def test_strides_of_one_token_or_head_are_not_used(m):
    """Views whose axis of one entry has a stride that is no multiple of 8."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    inv = torch.full((32,), 0.5, dtype=torch.float64, device="cuda")
    pos = torch.tensor([1000], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5], dtype=torch.int64, device="cuda")
    w, wq = bf16(512), bf16(128)
    kv, q = bf16(1, 576), bf16(1, 3, 128)
    got = []
    for kv_in, q_in in ((kv, q), (kv.as_strided((1, 576), (579, 1)), q.as_strided((1, 3, 128), (13, 128, 1)))):
        pool = torch.zeros((1, 64, 352), dtype=torch.uint8, device="cuda")
        out = m.mla_kv_norm_rope_append(kv_in, w, pos, inv, slots, pool, 1, 64, 64 * 352, q=q_in, q_weight=wq,
                                        q_out=torch.empty_like(q).as_strided((1, 3, 128), (3, 128, 1)))
        got.append((pool, out.clone()))
    k, pos = bf16(9, 1, 128), torch.arange(9, dtype=torch.int32, device="cuda")
    a, _ = m.mla_qk_norm_rope(k, None, pos, inv, q_weight=wq)
    b, _ = m.mla_qk_norm_rope(k.as_strided((9, 1, 128), (128, 3, 1)), None, pos, inv, q_weight=wq)
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], got[1][0]) and got[0][0].any()
    assert torch.equal(got[0][1], got[1][1]) and torch.equal(a, b)
