"""Dense decodes whose softmax weights span many binary orders: a first token far
above the rows that the output is made of, against float64 relative to those
rows."""
import math

import pytest
import torch

from dense_ref import LSE_TOL, ROW_BYTES, SCALE, attend64, random_pool, rows64, window_positions
from gpu_helpers import lib
from test_gpu_dense_decode import DEV, gen, lens_tensor, prefix_case, queries, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return lib()


def sink_case(g, fmt, lens, heads, bits, first):
    """(pool, stride, tables, blocks, queries): row 0 of table entry `first[b]` has no
    latent and a score `bits` binary orders above the others, whose scores
    differ by a few hundredths: the output is those rows' alone."""
    bt, spare, nb = tables(g, lens, extra_blocks=2)
    pool, stride = random_pool(g, nb, fmt)
    rows = pool.view(nb, 64, ROW_BYTES[fmt])
    rope = slice(ROW_BYTES[fmt] - 64, ROW_BYTES[fmt])
    rows[:, :, rope] = 0
    for block in first(bt, spare):
        rows[block, 0, :512 if fmt == 1 else 288] = 0
        rows[block, 0, ROW_BYTES[fmt] - 64] = 0x50  # e4m3 8.0
    qn, qr = queries(g, len(lens), 1, heads)
    qn *= 2.0 ** -10
    qr.zero_()
    qr[..., 0] = torch.linspace(bits, bits + 0.9, heads, device=DEV) / (8.0 * SCALE * math.log2(math.e))
    return pool, stride, bt, spare, nb, qn, qr


def assert_tail(out, lse, qn, qr, rows):
    """Against float64, relative to the rows that the output is made of.  Roundings
    as in out_tolerance, but no f16 partial; the weight of a row below 2^-23 of
    the largest is off by at most 2^-34 of that."""
    ref, rl, a = attend64(qn, qr, rows)
    v = rows[:, :512].abs().sum(0)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -9) * a + 2.0 ** -34 * v + 1e-30
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"{((err - tol) / (a + 1e-30)).max().item():.2e} of the weighted magnitude past it"
    assert (lse.double() - rl).abs().max() <= LSE_TOL


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bits", [16, 20, 24, 30])
def test_first_token_far_above_the_window(m, fmt, bits):
    """One slice a request: the window's rows, 16 to 30 binary orders below a
    first token whose latent is zero, keep their precision."""
    g = gen(50 + bits)
    lens = [600] * 170
    pool, stride, bt, _, nb, qn, qr = sink_case(g, fmt, lens, 64, bits, lambda bt, _: [int(b) for b in bt[:, 0]])
    assert m.mla_window_decode_workspace_size(170, 1, 64, bt.shape[1], 1, 300) == 0
    lse = torch.empty((170, 1, 64), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 1, 300, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    pos = torch.tensor(window_positions(600, 1, 0, 1, 300, 640), device=DEV)
    for b in (0, 50, 169):
        assert_tail(out[b, 0], lse[b, 0], qn[b, 0], qr[b, 0], rows64(pool, fmt, bt[b], pos))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bits", [16, 24])
def test_first_token_far_above_in_one_of_several_slices(m, fmt, bits):
    """The slice with that token keeps its other rows' part of the output, small
    as it is; so does a prefix that holds it."""
    g = gen(60 + bits)
    lens = [5000, 4000]
    pool, stride, bt, _, nb, qn, qr = sink_case(g, fmt, lens, 16, bits, lambda bt, _: [int(b) for b in bt[:, 0]])
    assert m.mla_window_decode_workspace_size(2, 1, 16, bt.shape[1], 0, 5000) > 0
    lse = torch.empty((2, 1, 16), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 0, 5000, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        rows = rows64(pool, fmt, bt[b], torch.arange(n, device=DEV))
        assert_tail(out[b, 0], lse[b, 0], qn[b, 0], qr[b, 0], rows)

    lens = [40, 0, 7]
    pool, stride, bt, pt, nb, qn, qr = sink_case(g, fmt, lens, 32, bits, lambda _, spare: [int(spare[0])])
    lse = torch.empty((3, 1, 32), device=DEV)
    out, _ = m.mla_prefix_decode(qn, qr, pool, stride, nb, pt, 100, bt, lens_tensor(lens), SCALE, 40, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    shared = rows64(pool, fmt, pt, torch.arange(100, device=DEV))
    for b, n in enumerate(lens):
        rows = torch.cat([shared, rows64(pool, fmt, bt[b], torch.arange(n, device=DEV))])
        assert_tail(out[b, 0], lse[b, 0], qn[b, 0], qr[b, 0], rows)


@pytest.mark.parametrize("fmt", [0, 1])
def test_wide_scores(m, fmt):
    """Scores with a deviation of 20 binary orders: maxima are raised in many tiles, of one column or another."""
    g = gen(70)
    lens = [1500, 700, 1501]
    bt, _, nb = tables(g, lens)
    pool, stride = random_pool(g, nb, fmt)
    qn, qr = queries(g, 3, 2, 64)
    qn, qr = qn * 8, qr * 8
    lse = torch.empty((3, 2, 64), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 4, 1400, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        for i in range(2):
            pos = torch.tensor(window_positions(n, 2, i, 4, 1400, bt.shape[1] * 64), device=DEV)
            rows = rows64(pool, fmt, bt[b], pos)
            ref, rl, a = attend64(qn[b, i], qr[b, i], rows)
            # a score's float accumulation: 576 x 2^-24 x the sum of |q k| scale, which
            # moves the LSE by at most itself and the output by twice that share of A;
            # weights 2^23 below the largest are off by at most 2^-34 of it, which counts
            # where the largest's value is 0
            v = rows[:, :512].abs().sum(0)
            q = torch.cat([qn[b, i], qr[b, i]], -1).double().abs()
            d = 576 * 2.0 ** -24 * (q @ rows.abs().t()).max().item() * SCALE
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * d) * a + 2.0 ** -34 * v
            assert ((out[b, i].double() - ref).abs() <= tol).all()
            assert (lse[b, i].double() - rl).abs().max() <= d + 2.0 ** -20


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("prefix,lens,q_len,heads", [(1, [3000, 5, 2500], 1, 16), (33, [9000], 2, 32),
                                                     (500, [2000] * 40, 1, 64)])
def test_prefix_much_shorter_than_the_own_rows(m, fmt, prefix, lens, q_len, heads):
    """The own rows have fewer slices than prefix-sized ones would be."""
    prefix_case(m, 80 + prefix, fmt, prefix, lens, q_len, heads)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("step", [0.0, 16.0])
@pytest.mark.parametrize("level", [2.0 ** 18, 1.5 * 2.0 ** 19, 2.0 ** 25, 2.0 ** 26, 1.25 * 2.0 ** 27, 2.0 ** 28])
def test_scores_whose_steps_are_coarse(m, fmt, step, level):
    """Scores of 2^18 to 2^28 (base 2), whose float steps reach 32: the last rows stand
    `step` above the others, and the output is a mean of rows, not an infinity."""
    g = gen(100)
    n = 200
    bt, _, nb = tables(g, [n])
    pool, stride = random_pool(g, nb, fmt)
    rows, rope = pool.view(nb, 64, ROW_BYTES[fmt]), ROW_BYTES[fmt] - 64
    rows[:, :, rope:] = 0
    rows[:, :, rope] = 0x38  # e4m3 1.0
    rows[bt[0, 2].long(), :, rope + 1] = 0x38
    rows[bt[0, 3].long(), :, rope + 1] = 0x38
    qn, qr = queries(g, 1, 1, 16)
    qn.zero_()
    qr.zero_()
    qr[..., 0], qr[..., 1] = level, step
    scale = math.log(2.0)  # a score is then q . k in base 2, but for the float of the two factors
    lse = torch.empty((1, 1, 16), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor([n]), scale, 0, n, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    v = rows64(pool, fmt, bt[0], torch.arange(n, device=DEV))[:, :512]
    got, h = out[0, 0].double(), 2.0 ** -24 * level
    # between the rows' least and largest values, whatever the steps make of the differences
    assert (got <= v.amax(0) * (1 + 2.0 ** -8) + 1e-6).all() and (got >= v.amin(0) * (1 + 2.0 ** -8) - 1e-6).all()
    if step == 0.0:
        # equal scores: P is the same power of two for every row of a slice.  Slices are
        # joined by float LSEs of this size, of which half a step is h: a slice's weight is
        # off by a factor of up to 2^h, and so is the sum it is divided by.
        tol = 2.0 ** -8 * v.mean(0).abs() + (2.0 ** (2 * h) - 1 + 2.0 ** -16) * v.abs().mean(0)
        assert ((got - v.mean(0)).abs() <= tol).all()
    # eight float roundings (the scale's factors and product, the score, the sum with log2 of the
    # denominator, ln 2 and its product), and a denominator of at most 200 x 2^16
    assert ((lse.double() / math.log(2.0) - level).abs() <= 8 * 2.0 ** -24 * level + 24).all()
