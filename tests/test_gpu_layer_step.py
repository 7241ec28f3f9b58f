"""The operators around the attention of a layer, run together: a decode step from the
residual's norm in 8 bits through 4-bit projections, the paged cache and the
window decode back to the residual's width; a prompt from norm and rotation to its
attention.  Each link is checked against float64 over what the link before gave;
the step is captured once and replayed.  And calls whose inputs are written late."""
import pytest
import torch

from dense_ref import SCALE
from gpu_helpers import lib
from test_gpu_add_norm_quant import check as check_norm
from test_gpu_fp4_matvec import check as check_product
from test_gpu_fp4_matvec import weights
from test_gpu_late_inputs import late_write  # noqa: F401
from test_gpu_norm_rope import INV
from test_gpu_prompt_attention import check as check_attention
from test_gpu_prompt_attention import starts
from test_gpu_serving_step import Server, check_append

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEADS, DIM = 32, 1024


@pytest.fixture(scope="module")
def m():
    return lib()


class Layer:
    """The 4-bit matrices of a layer beside the cache of a `Server`."""

    def __init__(self, m, batch, seed):
        self.m, g = m, torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.gen = g
        self.norm_w = (torch.randn(DIM, generator=g, device=DEV) * 0.1 + 1).to(torch.bfloat16)

        def matrix(*shape):
            codes, scales = weights(g, *shape)
            # scales near one: a product of k of them stays near the inputs' size
            scales = (torch.rand(scales.shape, generator=g, device=DEV) + 0.5).to(torch.float8_e4m3fn)
            return codes, scales, torch.full((shape[0],), shape[2] ** -0.5 / 3, device=DEV)

        self.to_q, self.to_kv = matrix(1, HEADS * 192, DIM), matrix(1, 576, DIM)
        self.up, self.down, self.back = matrix(HEADS, 512, 128), matrix(HEADS, 128, 512), matrix(1, DIM, HEADS * 128)
        self.server = Server(m, 0, batch, 64, 8, seed)
        self.server.q_w = self.server.bf16(192)

    def product(self, x, matrix, x_scales=None, out=None):
        codes, scales, ws = matrix
        if x.dim() == 2:
            codes, scales = codes[0], scales[0]
        return self.m.mla_fp4_matvec(x, codes, scales, ws, x_scales=x_scales, out=out)

    def step(self, x, residual, new):
        """One token a request; everything that is made on the way."""
        m, s, n = self.m, self.server, x.shape[0]
        codes, sc, residual = m.mla_add_norm_quant(x, self.norm_w, residual=residual)
        q = self.product(codes, self.to_q, sc).view(n, HEADS, 192)
        kv = self.product(codes, self.to_kv, sc)
        q_out, slots, pos, _ = s.append(kv, q, new, n)
        q_nope = self.product(q_out[..., :128], self.up).view(n, 1, HEADS, 512)
        q_rope = q_out[..., 128:].reshape(n, 1, HEADS, 64).contiguous()
        latent, _ = m.mla_window_decode(q_nope, q_rope, s.pool, s.stride, s.blocks, s.table, s.ctx, SCALE, 4, 200)
        heads = self.product(latent.view(n, HEADS, 512), self.down)
        y = self.product(heads.view(n, HEADS * 128), self.back)
        return dict(codes=codes, sc=sc, residual=residual, q=q, kv=kv, q_out=q_out, slots=slots, pos=pos, q_nope=q_nope,
                    latent=latent, heads=heads, y=y)


def inputs(layer, n):
    x = torch.randn((n, DIM), generator=layer.gen, device=DEV).to(torch.bfloat16)
    r = (torch.randn((n, DIM), generator=layer.gen, device=DEV) * 4).to(torch.bfloat16)
    return x, r


@pytest.mark.parametrize("batch", [1, 5, 24])
def test_decode_steps(m, batch):
    layer = Layer(m, batch, 11 + batch)
    new = torch.ones(batch, dtype=torch.int32, device=DEV)
    for _ in range(3):
        x, r = inputs(layer, batch)
        d = layer.step(x, r, new)
        torch.cuda.synchronize()
        check_norm(d["codes"], d["sc"], d["residual"], x, layer.norm_w, r, 128)
        a = d["codes"].view(batch, 1, DIM)
        check_product(d["q"].view(batch, 1, -1), a, d["sc"].view(batch, 1, -1), *layer.to_q)
        check_product(d["kv"].view(batch, 1, -1), a, d["sc"].view(batch, 1, -1), *layer.to_kv)
        check_append(layer.server, d["kv"], d["q"], d["q_out"], d["slots"], d["pos"])
        check_product(d["q_nope"].view(batch, HEADS, 512), d["q_out"][..., :128], None, *layer.up)
        check_product(d["heads"], d["latent"].view(batch, HEADS, 512), None, *layer.down)
        check_product(d["y"].view(batch, 1, -1), d["heads"].view(batch, 1, -1), None, *layer.back)
        assert d["y"].isfinite().all() and d["latent"].isfinite().all()


def test_captured_step(m):
    """A captured step replayed over advancing lengths gives what eager steps give."""
    batch = 6
    eager, replayed = Layer(m, batch, 5), Layer(m, batch, 5)
    new = torch.ones(batch, dtype=torch.int32, device=DEV)
    steps = [inputs(eager, batch) for _ in range(4)]
    x, r = steps[0][0].clone(), steps[0][1].clone()
    state = [t.clone() for t in (replayed.server.ctx, replayed.server.table, replayed.server.state, replayed.server.pool)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.step(x, r, new)  # nothing is set up for the first time while a graph is captured
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = replayed.step(x, r, new)
    for live, old in zip((replayed.server.ctx, replayed.server.table, replayed.server.state, replayed.server.pool), state):
        live.copy_(old)
    for a, b in steps:
        want = eager.step(a, b, new)
        x.copy_(a)
        r.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for name, t in want.items():
            assert torch.equal(out[name].view(torch.uint8), t.view(torch.uint8)), name


def test_prompts(m):
    """Two packed prompts: norm and rotation of queries and keys per head, then their attention."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    lens, heads, kv_heads = [300, 77], 8, 4
    n = sum(lens)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    q, kv, wq, wk = bf16(n, heads, 192), bf16(n, kv_heads, 192 + 128), bf16(192) * 0.2 + 1, bf16(192) * 0.2 + 1
    pos = torch.cat([torch.arange(x, device=DEV, dtype=torch.int32) for x in lens])
    k, v = kv[..., :192], kv[..., 192:]
    q2, k2 = m.mla_qk_norm_rope(q, k, pos, INV.to(DEV), q_weight=wq, k_weight=wk, rope_offset=128, k_out=k)
    at = starts(lens)
    lse = torch.empty((n, heads), device=DEV)
    out, _ = m.mla_prompt_attention(q2, k2, v, at, at, SCALE, lse=lse)
    check_attention(out, lse, q2, k2, v, at.tolist(), at.tolist(), SCALE, True)


def test_inputs_written_while_the_grid_waits(m, late_write):  # noqa: F811
    g = torch.Generator(device=DEV)
    g.manual_seed(8)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    # products: the tokens, their scales, the weights' codes and scales come late
    codes, scales = weights(g, 1, 700, 512)
    more = weights(g, 1, 700, 512)
    for tokens in (3, 20):
        x = [(torch.randn((tokens, 1, 512), generator=g, device=DEV) * 50).to(torch.float8_e4m3fn) for _ in range(2)]
        xs = [torch.rand((tokens, 1, 4), generator=g, device=DEV) for _ in range(2)]
        sets = [[x[0], xs[0], codes, scales], [x[1], xs[1], *more]]
        want = [m.mla_fp4_matvec(a, c, s, x_scales=b) for a, b, c, s in sets]
        live = [t.clone() for t in sets[0]]
        torch.cuda.synchronize()
        for step in range(8):
            k = (step + 1) % 2
            late_write(sets[k], live)
            got = m.mla_fp4_matvec(live[0], live[2], live[3], x_scales=live[1])
            torch.cuda.synchronize()
            assert torch.equal(got, want[k]), (tokens, step)
    # attention: queries, keys and values side by side, and the starts
    for q_lens, kv_lens in (([40, 60], [[300, 500], [450, 350]]), ([1, 3], [[3000, 5000], [4500, 3500]])):
        nq, nk = sum(q_lens), sum(kv_lens[0])
        q, kv = [bf16(nq, 4, 128) for _ in range(2)], [bf16(nk, 2, 256) for _ in range(2)]
        qs, ks = [starts(q_lens), starts(q_lens[::-1])], [starts(x) for x in kv_lens]

        def run(a, b, c, d):
            return m.mla_prompt_attention(a, b[..., :128], b[..., 128:], c, d, 0.1)[0]

        want = [run(q[k], kv[k], qs[k], ks[k]) for k in range(2)]
        live = [t.clone() for t in (q[0], kv[0], qs[0], ks[0])]
        torch.cuda.synchronize()
        for step in range(8):
            k = (step + 1) % 2
            late_write([q[k], kv[k], qs[k], ks[k]], live)
            got = run(*live)
            torch.cuda.synchronize()
            assert torch.equal(got, want[k]), (q_lens, step)
    assert m.mla_device_fault() == 0
