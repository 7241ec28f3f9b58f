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
