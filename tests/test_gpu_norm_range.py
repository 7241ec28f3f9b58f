"""The residual norm in 8 bits: every code against the exact quotient's rounding, and rows
at the end of float32's range.

A code is e4m3(y / s) with s = max|y| / 448 of its group.  The row's factor is a
power of two and a rest that meets the scales alone, so that y' = h 2^e w is off by
2^-24 of itself (h is the float32 sum), s by its own and the largest value's rounding,
the quotient by its own: together 4 x 2^-24.  Where the exact quotient is further than
2^-21 of itself from the middle between two neighbours the code is the exact one's."""
import pytest
import torch

from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRID = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def exact_codes(y, width):
    """(nearest e4m3 magnitude, whether the quotient is clear of a tie, group maxima)."""
    grid = GRID.to(DEV)
    n, d = y.shape
    groups = -(-d // width)
    parts = torch.nn.functional.pad(y.abs(), (0, groups * width - d)).view(n, groups, width)
    top = parts.amax(-1)
    q = (parts / (top / 448).clamp(min=1e-300)[..., None]).view(n, -1)[:, :d].contiguous()
    mid = (grid[1:] + grid[:-1]) / 2
    code = grid[torch.searchsorted(mid, q)]
    near = torch.searchsorted(mid, q).clamp(max=mid.numel() - 1)
    away = torch.minimum((q - mid[near]).abs(), (q - mid[(near - 1).clamp(min=0)]).abs())
    return code, away > 2.0 ** -21 * q, top


def check(m, x, w, r, group, eps):
    codes, scales, _ = m.mla_add_norm_quant(x, w, residual=r, group=group, eps=eps)
    h = x.double() if r is None else (x.float() + r.float()).double()
    rstd = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    width = group or x.shape[1]
    code, clear, top = exact_codes(h * w.double(), width)
    got = codes.float().double()
    assert torch.equal(got.abs()[clear], code[clear])
    # Few are left out: where weights are 1 and a row's largest is 1.75 x 2^k, all quotients of its 8-bit
    # values by 2^k / 256 have 8 bits, and of those one in 16 lies in the middle between two of 4 bits.
    assert (~clear).sum() <= max(2, clear.numel() // 8)
    assert ((got == 0) | (got.sign() == (h * w.double()).sign())).all()
    # each group's largest has the largest code
    whole = torch.nn.functional.pad(got.abs(), (0, top.shape[1] * width - got.shape[1])).view(*top.shape, width).amax(-1)
    assert (whole[top > 0] == 448).all() and (whole[top == 0] == 0).all()
    # the factor: 85 roundings of the sum of squares, rsqrt, three products
    want = top * rstd / 448
    assert ((scales.double() - want).abs() <= 2.0 ** -17 * want).all(), ((scales.double() - want).abs() / want).max()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 8), (40, 264), (64, 512), (50, 1544), (40, 4096), (300, 6144), (20, 16384)])
def test_codes_are_the_quotients(n, d, kind, group):
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(d + n)
    for scale in (1.0, 3e-5, 700.0):
        x = (torch.randn((n, d), generator=g, device=DEV) * scale).to(torch.bfloat16)
        w = (torch.randn(d, generator=g, device=DEV) * 0.3 + 1).to(torch.bfloat16)
        r = None if kind is None else (torch.randn((n, d), generator=g, device=DEV) * 3 * scale).to(kind)
        check(m, x, w, r, group, 1e-6)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [64, 2056, 6144, 16384])
@pytest.mark.parametrize("power", [60, 66, 100, 124])
def test_squares_past_float(power, d, group):
    """Rows whose squares leave float32's range, beside ordinary ones."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(d + power)
    x = (torch.randn((9, d), generator=g, device=DEV)).clamp(-7, 7)
    x[1::2] *= 2.0 ** power
    w = (torch.randn(d, generator=g, device=DEV) * 0.3 + 1).to(torch.bfloat16)
    check(m, x.to(torch.bfloat16), w, None, group, 1e-6)
    check(m, x.to(torch.bfloat16), w, x * 0.5, group, 1e-6)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("power,eps", [(66, 2.0 ** 130 * 2.0 ** -3), (64, 3e38), (62, 3.4e38), (50, 3.4e38), (64, 1e36)])
def test_eps_as_large_as_the_squares(power, eps, group):
    """eps counts beside squares past float32, and their sum with it may leave the range."""
    m = lib()
    g = torch.Generator(device=DEV)
    g.manual_seed(power)
    for d in (8, 512, 6152):
        x = (torch.randn((5, d), generator=g, device=DEV) * 2.0 ** power).to(torch.bfloat16)
        check(m, x, torch.ones(d, dtype=torch.bfloat16, device=DEV), None, group, eps)
