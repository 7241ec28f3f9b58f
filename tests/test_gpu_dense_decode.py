"""Dense decodes (sliding window with visible first tokens; shared prefix)
against float64 attention over the rows each query token sees."""
import math

import pytest
import torch

from dense_ref import (SCALE, assert_attention, attend64, random_pool, rows64, window_positions)
from gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    return lib()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def queries(g, *shape):
    return (torch.randn((*shape, 512), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((*shape, 64), generator=g, device=DEV).to(torch.bfloat16))


def tables(g, lens, extra_blocks=3, width=None):
    """Scattered block tables, -1 behind a request's last block."""
    need = [max(0, -(-n // 64)) for n in lens]
    total = sum(need) + extra_blocks
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((len(lens), width or max(1, *need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, perm[at:].contiguous(), total


def lens_tensor(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


def window_case(m, seed, fmt, lens, q_len, heads, sinks, window, stride=None, lse=True, scale=SCALE, **kw):
    g = gen(seed)
    bt, _, nb = tables(g, lens)
    pool, stride = random_pool(g, nb, fmt, stride)
    qn, qr = queries(g, len(lens), q_len, heads)
    lse_t = torch.full((len(lens), q_len, heads), float("nan"), device=DEV) if lse else None
    out, got = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), scale, sinks, window, fmt=fmt,
                                   lse=lse_t, **kw)
    torch.cuda.synchronize()
    assert m.mla_device_fault() == 0
    return dict(out=out, lse=got, qn=qn, qr=qr, pool=pool, stride=stride, bt=bt, nb=nb, lens=lens)


def check_window(c, fmt, q_len, sinks, window, scale=SCALE, only=None):
    held = c["bt"].shape[1] * 64
    for b, n in enumerate(c["lens"]):
        if only is not None and b not in only:
            continue
        for i in range(q_len):
            pos = torch.tensor(window_positions(n, q_len, i, sinks, window, held), device=DEV, dtype=torch.long)
            rows = rows64(c["pool"], fmt, c["bt"][b], pos)
            ref, lse, a = attend64(c["qn"][b, i], c["qr"][b, i], rows, scale)
            assert_attention(c["out"][b, i], c["lse"][b, i], ref, lse, a, f"request {b} token {i}")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("lens,q_len,heads,sinks,window", [
    ([1], 1, 16, 0, 1),                          # one row
    ([128], 1, 16, 0, 128),                      # one full tile
    ([129, 127, 64, 65, 0], 1, 16, 4, 1000),     # around a tile, an empty request
    ([500, 3, 77], 1, 16, 4, 100),               # sinks apart from the window
    ([500, 3, 101, 104, 105], 1, 48, 4, 100),    # sinks meet the window; 48 columns
    ([300, 2, 9], 4, 16, 4, 50),                 # four query tokens, one request shorter than them
    ([400, 290], 7, 32, 100, 33),                # 224 columns: groups of 64 and a rest of 32
    ([700], 3, 64, 0, 130),
    ([260, 40], 2, 128, 1, 64),
    ([4000, 1500], 1, 16, 64, 2000),             # several slices
    ([40, 41, 42], 15, 16, 200, 5),              # sinks beyond the context; 15 draft tokens
])
def test_window_decode(m, fmt, lens, q_len, heads, sinks, window):
    c = window_case(m, 11 + len(lens) * heads + q_len, fmt, lens, q_len, heads, sinks, window)
    check_window(c, fmt, q_len, sinks, window)


@pytest.mark.parametrize("fmt", [0, 1])
def test_window_many_groups(m, fmt):
    """More groups than SMs: one slice each, several waves."""
    lens = [1 + (37 * b) % 700 for b in range(200)]
    c = window_case(m, 5, fmt, lens, 1, 64, 4, 256)
    check_window(c, fmt, 1, 4, 256, only=range(0, 200, 17))


def test_window_split_into_one_per_sm(m):
    """One request over a long window: every SM has a slice, joined by the second kernel."""
    c = window_case(m, 6, 0, [30000], 1, 16, 4, 29000)
    check_window(c, 0, 1, 4, 29000)


@pytest.mark.parametrize("fmt,stride", [(0, 64 * 352 + 16), (0, 3 * 64 * 352), (1, 64 * 576 + 48)])
def test_window_padded_block_stride(m, fmt, stride):
    c = window_case(m, 7, fmt, [333, 100], 2, 16, 3, 200, stride=stride)
    check_window(c, fmt, 2, 3, 200)


def test_window_covers_context_equals_dense(m):
    """A window of 2^31 - 1 sees the whole context."""
    c = window_case(m, 8, 0, [777, 64], 2, 16, 0, 2 ** 31 - 1)
    check_window(c, 0, 2, 0, 2 ** 31 - 1)


def test_window_without_lse_and_with_own_buffers(m):
    g = gen(9)
    lens, q_len, heads = [900, 50], 2, 16
    bt, _, nb = tables(g, lens)
    pool, stride = random_pool(g, nb, 0)
    qn, qr = queries(g, 2, q_len, heads)
    need = m.mla_window_decode_workspace_size(2, q_len, heads, bt.shape[1], 4, 800)
    assert need > 0
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV)  # contents on entry do not matter
    out = torch.full((2, q_len, heads, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    a, none = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 4, 800, out=out,
                                  workspace=ws)
    assert none is None and a is out
    lse = torch.empty((2, q_len, heads), device=DEV)
    b, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 4, 800, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(a, b)  # and the same call twice gives the same bits


def test_window_bad_pages_are_not_seen(m):
    """Table entries outside the pool, and contexts longer than the table, lose
    their rows and nothing else."""
    g = gen(10)
    lens = [640, 640, 640]
    bt, _, nb = tables(g, lens, width=10)
    pool, stride = random_pool(g, nb, 0)
    qn, qr = queries(g, 3, 1, 16)
    bad = bt.clone()
    bad[0, 3], bad[0, 9], bad[1, :] = -1, nb, -7
    ctx = lens_tensor([640, 640, 2 ** 31 - 1])  # the third says far more than its table holds
    lse = torch.empty((3, 1, 16), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bad, ctx, SCALE, 600, 2 ** 31 - 1, lse=lse)
    torch.cuda.synchronize()
    assert m.mla_device_fault() == 0
    pos = torch.tensor([t for t in range(640) if t // 64 not in (3, 9)], device=DEV)
    ref, rl, a = attend64(qn[0, 0], qr[0, 0], rows64(pool, 0, bt[0], pos))
    assert_attention(out[0, 0], lse[0, 0], ref, rl, a)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    # 600 sinks, and the rows from position (2^31 - 1) - window on: 255 and later
    ref, rl, a = attend64(qn[2, 0], qr[2, 0], rows64(pool, 0, bt[2], torch.arange(640, device=DEV)))
    assert_attention(out[2, 0], lse[2, 0], ref, rl, a)


def test_window_nan_rows_reach_only_who_sees_them(m):
    """A NaN in a later draft token's row, in a row outside the window and in
    rows behind the context does not reach the tokens that do not see them; a
    token that does gets NaN."""
    g = gen(12)
    lens, q_len, heads = [300, 300], 4, 16
    for fmt in (0, 1):
        bt, _, nb = tables(g, lens)
        pool, stride = random_pool(g, nb, fmt)
        qn, qr = queries(g, 2, q_len, heads)
        rb = (352, 576)[fmt]

        def spoil(b, pos, byte):
            pool[bt[b, pos // 64].long(), pos % 64 * rb + byte] = 0x7F

        spoil(0, 299, 256 if fmt == 0 else 100)  # the last draft token: only token 3 sees it
        spoil(0, 150, rb - 1)                    # between the sinks and every window
        spoil(0, 301, 256 if fmt == 0 else 0)    # behind the context
        lse = torch.empty((2, q_len, heads), device=DEV)
        out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor(lens), SCALE, 4, 64, fmt=fmt, lse=lse)
        torch.cuda.synchronize()
        for b in range(2):
            for i in range(q_len):
                if b == 0 and i == 3:
                    assert torch.isnan(out[b, i]).all() and torch.isnan(lse[b, i]).all()
                    continue
                pos = torch.tensor(window_positions(300, q_len, i, 4, 64, 320), device=DEV)
                ref, rl, a = attend64(qn[b, i], qr[b, i], rows64(pool, fmt, bt[b], pos))
                assert_attention(out[b, i], lse[b, i], ref, rl, a, f"fmt {fmt} request {b} token {i}")


def test_nan_query_stays_with_its_head(m):
    g = gen(13)
    bt, _, nb = tables(g, [400])
    pool, stride = random_pool(g, nb, 0)
    qn, qr = queries(g, 1, 1, 32)
    qn[0, 0, 5, 17] = float("nan")
    qr[0, 0, 20, 3] = float("inf")
    lse = torch.empty((1, 1, 32), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor([400]), SCALE, 4, 300, lse=lse)
    torch.cuda.synchronize()
    pos = torch.tensor(window_positions(400, 1, 0, 4, 300, 448), device=DEV)
    ref, rl, a = attend64(qn[0, 0], qr[0, 0], rows64(pool, 0, bt[0], pos))
    good = [h for h in range(32) if h not in (5, 20)]
    assert_attention(out[0, 0][good], lse[0, 0][good], ref[good], rl[good], a[good])
    assert torch.isnan(out[0, 0, [5, 20]]).all() and torch.isnan(lse[0, 0, [5, 20]]).all()


@pytest.mark.parametrize("factor", [2.0 ** 40, 2.0 ** -40])
def test_query_range(m, factor):
    """Queries far outside FP16's range, the softmax scale undoing the factor (powers of two: exact)."""
    a = window_case(m, 14, 0, [300], 1, 16, 4, 200)
    lse = torch.empty((1, 1, 16), device=DEV)
    out, _ = m.mla_window_decode(a["qn"] * factor, a["qr"] * factor, a["pool"], a["stride"], a["nb"], a["bt"],
                                 lens_tensor([300]), SCALE / factor, 4, 200, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out, a["out"]) and torch.equal(lse, a["lse"])


def test_rising_scores_rescale(m):
    """Scores that rise by hundreds along the list: the maximum is raised tile after tile."""
    g = gen(15)
    n = 1024
    bt, _, nb = tables(g, [n])
    pool, stride = random_pool(g, nb, 1)
    rows = pool.view(nb, 64, 576)
    rope = torch.zeros((n, 64), device=DEV)
    rope[:, 0] = torch.arange(n, device=DEV) / 4.0  # e4m3 keeps about this slope
    for t in range(0, n, 64):
        rows[bt[0, t // 64].long(), :, 512:] = rope[t:t + 64].to(torch.float8_e4m3fn).view(torch.uint8)
    qn, qr = queries(g, 1, 1, 16)
    qr[..., 0] = 40.0
    lse = torch.empty((1, 1, 16), device=DEV)
    out, _ = m.mla_window_decode(qn, qr, pool, stride, nb, bt, lens_tensor([n]), SCALE, 0, n, fmt=1, lse=lse)
    torch.cuda.synchronize()
    ref, rl, a = attend64(qn[0, 0], qr[0, 0], rows64(pool, 1, bt[0], torch.arange(n, device=DEV)))
    # scores reach 740: their float accumulation is off by up to 576 x 2^-24 x 740, so
    # the LSE by 2.6e-2 and the output by twice that share of A
    d = 576 * 2.0 ** -24 * 740
    assert ((out[0, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2 * d) * a).all()
    assert (lse[0, 0].double() - rl).abs().max() <= d


# ------------------------------------------------------------------------ shared prefix
def prefix_case(m, seed, fmt, prefix, lens, q_len, heads, width=None, max_ctx=None):
    g = gen(seed)
    p = -(-prefix // 64)
    bt, spare, nb = tables(g, lens, extra_blocks=p + 2, width=width)
    pt = spare[:max(1, p)].contiguous()
    pool, stride = random_pool(g, nb, fmt)
    qn, qr = queries(g, len(lens), q_len, heads)
    lse = torch.full((len(lens), q_len, heads), float("nan"), device=DEV)
    out, _ = m.mla_prefix_decode(qn, qr, pool, stride, nb, pt, prefix, bt, lens_tensor(lens), SCALE,
                                 max(lens) if max_ctx is None else max_ctx, fmt=fmt, lse=lse)
    torch.cuda.synchronize()
    assert m.mla_device_fault() == 0
    shared = rows64(pool, fmt, pt, torch.arange(prefix, device=DEV))
    for b, n in enumerate(lens):
        n = n if max_ctx is None else min(n, max_ctx)
        for i in range(q_len):
            own = rows64(pool, fmt, bt[b], torch.arange(max(0, n - q_len + i + 1), device=DEV))
            ref, rl, a = attend64(qn[b, i], qr[b, i], torch.cat([shared, own]))
            assert_attention(out[b, i], lse[b, i], ref, rl, a, f"request {b} token {i}")


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("prefix,lens,q_len,heads", [
    (1, [1], 1, 16),
    (128, [1, 1], 1, 16),
    (1000, [0, 5, 200], 1, 16),           # 48 columns over the prefix; a request with nothing of its own
    (129, [3, 70, 1, 64, 65], 2, 16),     # 160 columns: 64, 64, 32
    (5000, [300] * 9, 1, 32),
    (64, [130, 2], 3, 64),
    (777, [0, 0], 1, 128),
    (0, [100, 0, 33], 1, 16),             # no prefix: own rows alone
    (300, [2, 1, 0], 4, 16),              # fewer own tokens than query tokens
])
def test_prefix_decode(m, fmt, prefix, lens, q_len, heads):
    prefix_case(m, prefix + len(lens), fmt, prefix, lens, q_len, heads)


def test_prefix_decode_long(m):
    prefix_case(m, 21, 0, 20000, [700, 1, 64, 300] * 4, 1, 16)


def test_prefix_wide_table_and_cut_contexts(m):
    """A table wider than the contexts, and contexts longer than max_context_len."""
    prefix_case(m, 22, 0, 200, [100, 90], 1, 16, width=40)
    prefix_case(m, 23, 1, 200, [100, 90], 1, 16, max_ctx=64)


def test_prefix_equals_window_over_joined_tables(m):
    """The same rows as one context: both decodes answer within their tolerance of the same reference."""
    g = gen(24)
    prefix, lens = 640, [100, 37]  # a whole number of blocks, so one table can name both parts
    bt, spare, nb = tables(g, lens, extra_blocks=10)
    pool, stride = random_pool(g, nb, 0)
    qn, qr = queries(g, 2, 1, 16)
    la, lb = torch.empty((2, 1, 16), device=DEV), torch.empty((2, 1, 16), device=DEV)
    a, _ = m.mla_prefix_decode(qn, qr, pool, stride, nb, spare, prefix, bt, lens_tensor(lens), SCALE, 100, lse=la)
    joined = torch.cat([spare.expand(2, -1), bt], 1).contiguous()
    b, _ = m.mla_window_decode(qn, qr, pool, stride, nb, joined, lens_tensor([prefix + n for n in lens]), SCALE, 0,
                               10 ** 6, lse=lb)
    torch.cuda.synchronize()
    for r, n in enumerate(lens):
        ref, rl, w = attend64(qn[r, 0], qr[r, 0], rows64(pool, 0, joined[r], torch.arange(prefix + n, device=DEV)))
        assert_attention(a[r, 0], la[r, 0], ref, rl, w)
        assert_attention(b[r, 0], lb[r, 0], ref, rl, w)


# ------------------------------------------------------------------------ use
def test_two_streams_and_a_graph(m):
    """Two calls at once on streams of their own, and a captured call replayed on new data."""
    g = gen(31)
    lens = [900, 300, 77]
    bt, _, nb = tables(g, lens)
    pool, stride = random_pool(g, nb, 0)
    ctx = lens_tensor(lens)
    q1, q2 = queries(g, 3, 1, 16), queries(g, 3, 2, 32)
    want1, _ = m.mla_window_decode(*q1, pool, stride, nb, bt, ctx, SCALE, 4, 500)
    want2, _ = m.mla_prefix_decode(*q2, pool, stride, nb, bt[0], 500, bt, ctx, SCALE, 900)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        a, _ = m.mla_window_decode(*q1, pool, stride, nb, bt, ctx, SCALE, 4, 500, stream=s1)
        b, _ = m.mla_prefix_decode(*q2, pool, stride, nb, bt[0], 500, bt, ctx, SCALE, 900, stream=s2)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want1) and torch.equal(b, want2)

    qn, qr = q1[0].clone(), q1[1].clone()
    out = torch.empty_like(want1)
    ws = torch.empty(m.mla_window_decode_workspace_size(3, 1, 16, bt.shape[1], 4, 500), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mla_window_decode(qn, qr, pool, stride, nb, bt, ctx, SCALE, 4, 500, out=out, workspace=ws)
    for seed in (1, 2):
        new = queries(gen(seed), 3, 1, 16)
        qn.copy_(new[0])
        qr.copy_(new[1])
        graph.replay()
        want, _ = m.mla_window_decode(*new, pool, stride, nb, bt, ctx, SCALE, 4, 500)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals(m):
    g = gen(41)
    bt, _, nb = tables(g, [100])
    pool, stride = random_pool(g, nb, 0)
    qn, qr = queries(g, 1, 1, 16)
    ctx = lens_tensor([100])
    args = (qn, qr, pool, stride, nb, bt, ctx, SCALE)
    for bad in (dict(sinks=-1, window=5), dict(sinks=0, window=0)):
        with pytest.raises(m.MlaError):
            m.mla_window_decode(*args, **bad)
    with pytest.raises(m.MlaError):
        m.mla_window_decode(*args[:7], math.nan, 0, 5)
    with pytest.raises(m.MlaError):
        m.mla_window_decode(*args, 0, 5, block_size=32)
    with pytest.raises(m.MlaError):
        m.mla_window_decode(qn[:, :, :8].contiguous(), qr[:, :, :8].contiguous(), *args[2:], 0, 5)
    with pytest.raises(ValueError):
        m.mla_window_decode(qn, qr, pool, stride, nb + 10, bt, ctx, SCALE, 0, 5)  # pool too small
    with pytest.raises(ValueError):
        m.mla_window_decode(*args, 0, 5, out=torch.empty((1, 1, 16, 256), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        m.mla_window_decode(qn.cpu(), qr, *args[2:], 0, 5)
    big = tables(g, [5000])
    with pytest.raises(m.MlaError):  # workspace too small
        m.mla_window_decode(qn, qr, pool, stride, nb, big[0], ctx, SCALE, 0, 5000,
                            workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        m.mla_prefix_decode(qn, qr, pool, stride, nb, bt[0], 64 * bt.shape[1] + 1, bt, ctx, SCALE, 100)
    with pytest.raises(m.MlaError):
        m.mla_prefix_decode(qn, qr, pool, stride, nb, bt[0], -1, bt, ctx, SCALE, 100)
    e = torch.empty((0, 1, 16, 512), dtype=torch.bfloat16, device=DEV)
    out, _ = m.mla_window_decode(e, e[..., :64].contiguous(), pool, stride, nb, bt[:0], ctx[:0], SCALE, 0, 5)
    assert out.shape == (0, 1, 16, 512)
