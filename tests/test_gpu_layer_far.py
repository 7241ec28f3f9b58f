"""The operators around the attention of a layer where offsets pass 32 bits, and
called at the same time on several streams."""
import pytest
import torch

from gpu_helpers import lib
from test_gpu_add_norm_quant import check as check_norm
from test_gpu_fp4_matvec import check as check_product
from test_gpu_layer_step import Layer, inputs
from test_gpu_prompt_attention import bf16, starts
from test_gpu_prompt_attention import check as check_attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    yield lib()
    torch.cuda.empty_cache()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def far(values, stride):
    """`values` [rows, ...] with its rows `stride` elements apart."""
    t = torch.empty((values.shape[0] - 1) * stride + values[0].numel(), dtype=values.dtype, device=DEV)
    t = t.as_strided(values.shape, (stride, *values[0].stride()))
    return t.copy_(values)


@pytest.mark.parametrize("q_lens,kv_lens", [([40], [40]), ([2, 1], [30, 10])])
def test_attention(m, q_lens, kv_lens):
    g = gen(1)
    q, k, v = bf16(g, sum(q_lens), 2, 128), bf16(g, 40, 2, 128), bf16(g, 40, 2, 128)
    step = 2 ** 26  # 40 of them are 2^31.3
    qs, ks = starts(q_lens), starts(kv_lens)
    out = far(torch.zeros_like(q), step)
    kv = far(torch.cat([k, v], 2), step)
    m.mla_prompt_attention(far(q, step), kv[..., :128], kv[..., 128:], qs, ks, 0.1, out=out)
    check_attention(out, None, q, k, v, qs.tolist(), ks.tolist(), 0.1, True)
    # an infinity in the last token's values is seen by the last query alone
    kv[-1, 1, 128:] = float("inf")
    again = far(torch.zeros_like(q), step)
    m.mla_prompt_attention(far(q, step), kv[..., :128], kv[..., 128:], qs, ks, 0.1, out=again)
    assert (again[-1, 1] == float("inf")).all()
    again[-1, 1] = out[-1, 1]
    assert torch.equal(again, out)


def test_norm(m):
    g = gen(2)
    x, r = bf16(g, 3, 1024), torch.randn((3, 1024), generator=g, device=DEV)
    w = bf16(g, 1024)
    step = 2 ** 30 + 8
    wide = far(r, step)
    codes, scales, h = m.mla_add_norm_quant(far(x, step), w, residual=wide, residual_out=wide)
    check_norm(codes, scales, h, x, w, r, 128)


def test_products(m):
    g = gen(3)
    n, k, tokens = 360_000, 12_288, 3
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(0, 127, (n, k // 16), generator=g, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert codes.numel() > 2 ** 31
    x = bf16(g, tokens, k)
    out = far(torch.zeros((tokens, n), device=DEV), 2 ** 30 + 8)
    m.mla_fp4_matvec(far(x, 2 ** 30 + 8), codes, scales, out=out)
    for rows in (slice(0, 100), slice(n // 2, n // 2 + 100), slice(n - 100, n)):
        check_product(out[:, None, rows], x[:, None], None, codes[None, rows], scales[None, rows], None)


def test_calls_at_once(m):
    """Prompts, a decode step and products on streams of their own, none waiting for another."""
    g = gen(4)
    layer = Layer(m, 4, 9)
    at, more = starts([1500, 700]), starts([3, 1])
    q, kv = bf16(g, 2200, 8, 192), bf16(g, 2200, 4, 320)
    few, long_at = bf16(g, 4, 8, 192), starts([9000, 5000])
    long_kv = bf16(g, 14000, 4, 320)
    x, r = inputs(layer, 4)
    norm_x, norm_w = bf16(g, 3000, 2048), bf16(g, 2048)
    y = bf16(g, 32, 1024)
    step_codes, step_scales, _ = layer.to_q

    def prompt():
        return [m.mla_prompt_attention(q, kv[..., :192], kv[..., 192:], at, at, 0.1)[0]]

    def drafts():
        return [m.mla_prompt_attention(few, long_kv[..., :192], long_kv[..., 192:], more, long_at, 0.1)[0]]

    def norm():
        return list(m.mla_add_norm_quant(norm_x, norm_w))[:2]

    def product():
        return [m.mla_fp4_matvec(y, step_codes[0], step_scales[0])]

    def link():
        s, rq = layer.server, x.shape[0]
        q_nope = layer.product(q[:rq].repeat(1, 4, 1)[..., :128], layer.up).view(rq, 1, 32, 512)
        q_rope = q[:rq].repeat(1, 4, 1)[..., 128:].reshape(rq, 1, 32, 64).contiguous()
        return [m.mla_window_decode(q_nope, q_rope, s.pool, s.stride, s.blocks, s.table, s.ctx, 0.1, 4, 200)[0]]

    for _ in range(3):  # a few tokens in the cache
        layer.step(x, r, torch.ones(4, dtype=torch.int32, device=DEV))
    calls = [prompt, drafts, norm, product, link]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(15):
        for i, (f, stream) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(stream):
                got[i].append(f())
    torch.cuda.synchronize()
    for i, (w, runs) in enumerate(zip(want, got)):
        for run in runs:
            for a, b in zip(w, run):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), calls[i].__name__
    assert m.mla_device_fault() == 0
