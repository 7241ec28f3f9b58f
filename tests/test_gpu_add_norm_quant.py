"""Residual's addition, norm and 8-bit output against float64.

Tolerances.  The kernel's y is float32: the sum of squares of n values (at most
16,384 in a tree of 8 chunks x 8 values a lane, five shuffles and 16 warps: 85
roundings in a row, all of one sign, 85 x 2^-24), rsqrt (2 units), three products
and the sum h (2^-24 of |x| + |r|): DELTA = 2^-17 of |y| covers them, apart from
what cancels in h, which is a term of its own.  A code is off by half a step: 2^-4
of the value, or 2^-10 of the scale below e4m3's normal range."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DELTA = 2.0 ** -17
EPS = 1e-6


def rows(g, n, d, scale=1.0, dtype=torch.bfloat16, pad=0):
    t = (torch.randn((n, d + pad), generator=g, device=DEV) * scale).to(dtype)
    return t[:, :d]


def reference(x, w, r, eps):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w.double()
    slack = torch.zeros_like(h) if r is None else 2.0 ** -24 * (x.double().abs() + r.double().abs())
    return h, y, slack / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w.double().abs()


def check(codes, scales, h_out, x, w, r, group, eps=EPS):
    h, y, slack = reference(x, w, r, eps)
    n, d = y.shape
    width = d if group == 0 else group
    top = torch.stack([p.abs().amax(-1) for p in y.split(width, 1)], 1)
    most = torch.stack([p.amax(-1) for p in slack.split(width, 1)], 1)
    assert scales.shape == top.shape
    assert ((scales.double() - top / 448).abs() <= (DELTA * top + most) / 448).all()
    s = scales.double().repeat_interleave(width, 1)[:, :d]
    err = (codes.float().double() * s - y).abs()
    assert (err <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s + 2 * DELTA * y.abs() + 2 * slack).all()
    # no value is a step further than the nearest: the codes fill their range
    assert (codes.float().abs().amax(1) >= 416).all()
    if r is None:
        assert h_out is None
    else:
        step = 2.0 ** -8 if h_out.dtype == torch.bfloat16 else 2.0 ** -24
        assert h_out.dtype == r.dtype
        assert ((h_out.double() - h).abs() <= step * 1.01 * h.abs() + 2.0 ** -23 * (x.double().abs() + r.double().abs())).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 136), (5, 256), (2, 264), (1, 512), (7, 520), (33, 1024), (9, 1544),
                                 (1, 2048), (1300, 2056), (17, 4096), (1, 4104), (700, 6144), (5, 6152), (3, 8192),
                                 (2, 8200), (11, 16384)])
def test_sizes(n, d, kind, group):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(n * 31 + d)
    x, w = rows(g, n, d), (torch.randn(d, generator=g, device=DEV) * 0.3 + 1).to(torch.bfloat16)
    r = None if kind is None else rows(g, n, d, 3.0, kind)
    codes, scales, h = m.mla_add_norm_quant(x, w, residual=r, group=group)
    check(codes, scales, h, x, w, r, group)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_strides_and_place(kind):
    """Strided rows, outputs in larger buffers whose other elements stay, the residual in place."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    n, d = 37, 1544
    x, w = rows(g, n, d, pad=24), rows(g, 1, d)[0].contiguous()
    r = rows(g, n, d, 2.0, kind, pad=8)
    keep = r.clone()
    beside = r.as_strided((n, 8), r.stride(), r.storage_offset() + d).clone()
    codes, scales, h = m.mla_add_norm_quant(x, w, residual=r, residual_out=r)
    assert h is r
    check(codes, scales, h, x, w, keep, 128)
    assert torch.equal(beside, r.as_strided((n, 8), r.stride(), r.storage_offset() + d))
    room_c = torch.full((n + 2, d), 0x55, dtype=torch.uint8, device=DEV)
    room_s = torch.full((n + 2, 13), -7.0, device=DEV)
    out = torch.full((n + 2, d + 16), 5.0, dtype=kind, device=DEV)
    got = m.mla_add_norm_quant(x, w, residual=keep, codes=room_c[1:n + 1], scales=room_s[1:n + 1],
                               residual_out=out[1:n + 1, :d])
    assert torch.equal(got[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got[1], scales)
    assert torch.equal(got[2], h)
    assert (room_c[0] == 0x55).all() and (room_c[-1] == 0x55).all()
    assert (room_s[0] == -7).all() and (room_s[-1] == -7).all()
    assert (out[0] == 5).all() and (out[-1] == 5).all() and (out[:, d:] == 5).all()


def test_rows_without_numbers():
    """Zeros, infinities, NaN, squares past float32 and values below its normal range, beside ordinary rows."""
    m = lib()
    n, d = 9, 512
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = rows(g, n, d).clone()
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    x[1] = 0
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    x[4] *= 2.0 ** 100
    x[5] *= 2.0 ** -120
    x[6, 256:384] = 0
    for group in (128, 0):
        codes, scales, _ = m.mla_add_norm_quant(x, w, group=group, eps=1e-30)
        plain = [0, 4, 6, 7, 8]
        check(codes[plain], scales[plain], None, x[plain], w, None, group, 1e-30)
        assert (codes[1].float() == 0).all() and (scales[1] == 0).all()
        assert codes[2].float().isnan().all() and scales[2].isnan().all()
        assert codes[3, 5].float().isnan() and scales[3, 0].isnan()
        if group:
            assert (scales[3, 1:] == 0).all() and (codes[3, 128:].float() == 0).all()
            assert scales[6, 2] == 0 and (codes[6, 256:384].float() == 0).all()
    # a row whose scales are below float32's normal range
    tiny = (torch.ones(1, d, device=DEV)).to(torch.bfloat16)
    w2 = torch.full((d,), 2.0 ** -126, dtype=torch.bfloat16, device=DEV)
    codes, scales, _ = m.mla_add_norm_quant(tiny, w2)
    # half a step of a subnormal scale: 2^-150 of 2^-126 / 448 is 2^-15.2
    assert ((codes.float().double() * scales.double().repeat_interleave(128, 1) / 2.0 ** -126 - 1).abs() <= 2.0 ** -4 + 2.0 ** -15).all()


def test_zero_rows_and_refusals():
    m = lib()
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = torch.ones((4, 64), dtype=torch.bfloat16, device=DEV)
    codes, scales, h = m.mla_add_norm_quant(x[:0], w, residual=x[:0])
    assert codes.shape == (0, 64) and scales.shape == (0, 1) and h.shape == (0, 64)
    with pytest.raises(TypeError):
        m.mla_add_norm_quant(x.float(), w)
    with pytest.raises(TypeError):
        m.mla_add_norm_quant(x, w, residual=x.half())
    with pytest.raises(ValueError):
        m.mla_add_norm_quant(x, w[:32])
    with pytest.raises(ValueError):
        m.mla_add_norm_quant(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        m.mla_add_norm_quant(x.t(), w[:4])
    with pytest.raises(m.MlaError):
        m.mla_add_norm_quant(x, w, group=64)
    with pytest.raises(ValueError):
        m.mla_add_norm_quant(x.cpu(), w)


def test_captured_and_on_another_stream():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    n, d = 50, 6144
    x, w, r = rows(g, n, d), rows(g, 1, d)[0].contiguous(), rows(g, n, d, 2.0)
    want = m.mla_add_norm_quant(x, w, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.mla_add_norm_quant(x, w, residual=r, stream=side)
    side.synchronize()
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mla_add_norm_quant(x, w, residual=r, codes=outs[0], scales=outs[1], residual_out=outs[2])
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
