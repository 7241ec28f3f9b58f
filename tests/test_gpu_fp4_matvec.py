"""Products with 4-bit weights against float64.

Tolerances.  Operands are exact, so what is lost is the sums': of each 128
products in the tensor core (8 steps of 16, each with its terms cut to float32's
step at the largest of them: at most 2^-22 of the sum of their magnitudes a step,
8 of them), of the pieces, warps and CTAs (one float32 addition each), and of a
bf16 x 2^-39 of the largest of its 128.  With A = sum |x w|, N pieces of 128:
(8 x 2^-22 + (N + 80) x 2^-24) A, the rounding of out (2^-8 or 2^-24), and the two
factors' (2^-23)."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(codes):
    """What e2m1 codes [..., K / 2] stand for, in float64 [..., K]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]


def weights(g, groups, n, k):
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    # every finite scale, the subnormal ones among them
    scales = torch.randint(0, 127, (groups, n, k // 16), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales.view(torch.float8_e4m3fn)


def inputs(g, kind, tokens, groups, k, per_row=False):
    if kind == "bf16":
        x = torch.randn((tokens, groups, k), generator=g, device=DEV)
        x *= torch.exp2(torch.randint(-30, 30, (tokens, groups, 1), generator=g, device=DEV).float())
        return x.to(torch.bfloat16), None
    x = (torch.randn((tokens, groups, k), generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x, torch.rand((tokens, groups, 1 if per_row else -(-k // 128)), generator=g, device=DEV) + 0.01


def check(y, x, x_scales, codes, scales, ws):
    k = x.shape[-1]
    xd = x.float().double()
    if x_scales is not None:
        xd = xd * x_scales.double().repeat_interleave(128 if x_scales.shape[-1] > 1 else k, -1)[..., :k]
    w = values(codes) * scales.float().double().repeat_interleave(16, -1)
    if ws is not None:
        w = w * ws.double()[:, None, None]
    want = torch.einsum("tgk,gnk->tgn", xd, w)
    mag = torch.einsum("tgk,gnk->tgn", xd.abs(), w.abs())
    top = torch.stack([p.abs().amax(-1) for p in xd.split(128, -1)], -1).repeat_interleave(128, -1)[..., :k]
    lost = torch.einsum("tgk,gnk->tgn", top, w.abs()) * 2.0 ** -39 if x_scales is None else 0
    pieces = -(-k // 128)
    out_step = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (8 * 2.0 ** -22 + (pieces + 80) * 2.0 ** -24 + 2.0 ** -23) * mag + lost + out_step * want.abs() * 1.01
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (err - tol).max().item()


SIZES = [(1, 1, 1, 32), (1, 1, 17, 64), (3, 1, 130, 160), (8, 1, 2001, 1504), (9, 1, 300, 4128), (16, 1, 64, 512),
         (17, 1, 1000, 2080), (32, 2, 129, 96), (33, 1, 77, 128), (64, 3, 40, 416), (5, 64, 31, 128), (1, 1, 6144, 6144),
         (1, 1, 3, 16384), (4, 16, 512, 128), (32, 16, 128, 512), (70, 1, 257, 1056), (2, 1, 20011, 256)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_rows"])
@pytest.mark.parametrize("tokens,groups,n,k", SIZES)
def test_sizes(tokens, groups, n, k, kind, out):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens * 7 + n + k)
    codes, scales = weights(g, groups, n, k)
    x, xs = inputs(g, kind[:4], tokens, groups, k, kind == "e4m3_rows")
    ws = torch.rand(groups, generator=g, device=DEV) * 2 ** -7 + 2 ** -9
    y = m.mla_fp4_matvec(x, codes, scales, ws, x_scales=xs, out_dtype=out)
    assert y.shape == (tokens, groups, n) and y.dtype == out
    check(y, x, xs, codes, scales, ws)
    again = m.mla_fp4_matvec(x, codes, scales, ws, x_scales=xs, out_dtype=out)
    assert torch.equal(y, again)


def test_one_matrix_and_strides():
    """[T, K] with one matrix; a slice of the heads' dims as x, out in a larger buffer."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    codes, scales = weights(g, 4, 50, 128)
    wide = torch.randn((6, 4, 192), generator=g, device=DEV).to(torch.bfloat16)
    x = wide[..., :128]
    room = torch.full((6, 4, 71), 9.0, device=DEV)
    y = m.mla_fp4_matvec(x, codes, scales, out=room[..., 11:61])
    check(y, x, None, codes, scales, None)
    assert (room[..., :11] == 9).all() and (room[..., 61:] == 9).all()
    turned = m.mla_fp4_matvec(x.transpose(0, 1).contiguous().transpose(0, 1), codes, scales, out_dtype=torch.float32)
    assert torch.equal(turned, y)
    one = m.mla_fp4_matvec(x[:, 1], codes[1], scales[1], out_dtype=torch.float32)
    assert torch.equal(one, y[:, 1])
    assert m.mla_fp4_matvec(x[:0], codes, scales).shape == (0, 4, 50)
    assert m.mla_fp4_matvec(x[:, 1], codes[1, :0], scales[1, :0]).shape == (6, 0)
    scales_u8 = m.mla_fp4_matvec(x, codes, scales.view(torch.uint8), out_dtype=torch.float32)
    assert torch.equal(scales_u8, y)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_tokens_and_rows_do_not_touch_each_other(kind):
    """NaN and infinities of one token or weight row stay there."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    codes, scales = weights(g, 1, 40, 256)
    x, xs = inputs(g, kind, 12, 1, 256)
    want = m.mla_fp4_matvec(x, codes, scales, x_scales=xs, out_dtype=torch.float32)
    x = x.clone()
    x[3, 0, 130] = float("nan")
    if kind == "bf16":
        x[5, 0, 7] = float("inf")
    scales = scales.clone()
    scales.view(torch.uint8)[0, 9, 3] = 0x7F  # NaN
    y = m.mla_fp4_matvec(x, codes, scales, x_scales=xs, out_dtype=torch.float32)
    assert y[3].isnan().all() and y[:, 0, 9].isnan().all()
    if kind == "bf16":
        assert not y[5].isfinite().any()
    tokens, rows = [t for t in range(12) if t not in (3, 5)], [n for n in range(40) if n != 9]
    assert torch.equal(y[tokens][:, 0, rows], want[tokens][:, 0, rows])
    # x far below or above f16's range
    x = torch.full((2, 64), 2.0 ** -126, dtype=torch.bfloat16, device=DEV)
    x[1] = 2.0 ** 120
    c = torch.full((1, 32), 0x22, dtype=torch.uint8, device=DEV)  # 1, 1
    s = torch.full((1, 4), 1.0, device=DEV).to(torch.float8_e4m3fn)
    assert m.mla_fp4_matvec(x, c, s, out_dtype=torch.float32).flatten().tolist() == [2.0 ** -120, 2.0 ** 126]


def test_streams_and_capture():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    codes, scales = weights(g, 1, 1000, 2048)
    x, xs = inputs(g, "e4m3", 20, 1, 2048)
    want = m.mla_fp4_matvec(x, codes, scales, x_scales=xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.mla_fp4_matvec(x, codes, scales, x_scales=xs, stream=side)
    side.synchronize()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mla_fp4_matvec(x, codes, scales, x_scales=xs, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(want, out)


def test_refusals():
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    codes, scales = weights(g, 1, 8, 64)
    x, xs = inputs(g, "e4m3", 2, 1, 64)
    b = x.float().to(torch.bfloat16)
    for bad in (lambda: m.mla_fp4_matvec(x, codes, scales), lambda: m.mla_fp4_matvec(b, codes, scales, x_scales=xs),
                lambda: m.mla_fp4_matvec(b, codes[:, :, :16], scales), lambda: m.mla_fp4_matvec(b[:, 0], codes, scales),
                lambda: m.mla_fp4_matvec(b, codes, scales[:, :4]), lambda: m.mla_fp4_matvec(b, codes, scales, xs.flatten()),
                lambda: m.mla_fp4_matvec(b, codes, scales, out=torch.empty((2, 1, 9), device=DEV)),
                lambda: m.mla_fp4_matvec(b.cpu(), codes, scales)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.mla_fp4_matvec(b.float(), codes, scales), lambda: m.mla_fp4_matvec(b, codes.float(), scales),
                lambda: m.mla_fp4_matvec(b, codes, scales.float()),
                lambda: m.mla_fp4_matvec(b, codes, scales, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(m.MlaError):  # k = 48
        m.mla_fp4_matvec(b[..., :48], codes[..., :24].contiguous(), scales[..., :3].contiguous())
    with pytest.raises(m.MlaError):  # rows of out that overlap
        m.mla_fp4_matvec(b, codes, scales, out=torch.empty(64, device=DEV).as_strided((2, 1, 8), (4, 8, 1)))


@pytest.mark.parametrize("kind,tokens,groups,n,k", [("bf16", 4096, 1, 1001, 16384), ("e4m3", 4096, 1, 1001, 25632),
                                                    ("e4m3", 9, 300, 1048, 8192), ("bf16", 1, 4, 70000, 96)])
def test_more_sums_than_fit_beside_the_tokens(kind, tokens, groups, n, k):
    """Many rows of many tokens a CTA, or of many matrices: their sums leave the tokens
    little room in shared memory, and CTAs come in rounds."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    codes, scales = weights(g, groups, n, k)
    x, xs = inputs(g, kind, tokens, groups, k)
    y = m.mla_fp4_matvec(x, codes, scales, x_scales=xs, out_dtype=torch.float32)
    for t in range(0, tokens, 1024):  # the comparison's memory
        part = slice(t, t + 1024)
        for j in range(0, groups, 30):
            of = slice(j, j + 30)
            check(y[part, of], x[part, of], None if xs is None else xs[part, of], codes[of], scales[of], None)


def test_one_token_for_all_matrices():
    """x with a stride of 0 over the groups."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    codes, scales = weights(g, 5, 200, 352)
    for kind in ("bf16", "e4m3"):
        x, xs = inputs(g, kind, 3, 1, 352)
        wide = x.expand(3, 5, 352)
        xs = None if xs is None else xs.expand(3, 5, 3).contiguous()
        y = m.mla_fp4_matvec(wide, codes, scales, x_scales=xs, out_dtype=torch.float32)
        check(y, wide, xs, codes, scales, None)
