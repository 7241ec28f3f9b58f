"""The operators around the cache run together as a serving step: block tables
from the lengths, norm and rotation into the cache with the queries', then the
decode that reads those rows.  Checked link by link against float64 forms, and
captured once and replayed."""
import numpy as np
import pytest
import torch

import oracle as O
from dense_ref import (ROW_BYTES, SCALE, assert_attention, attend64, extend_loop, rows64, window_positions)
from gpu_helpers import lib, u16
from test_gpu_norm_rope import EPS, INV, assert_heads, heads64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEADS, NOPE = 16, 128  # a head's query: 128 values that meet the latent through w_uk, 64 that are rotated


@pytest.fixture(scope="module")
def m():
    return lib()


class Server:
    """Weights, the paged cache, and the state of a batch of requests on the device."""

    def __init__(self, m, fmt, batch, blocks, width, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.m, self.fmt, self.batch, self.blocks, self.gen = m, fmt, batch, blocks, g
        self.stride = 64 * ROW_BYTES[fmt]
        self.pool = torch.full((blocks, self.stride), 0x7F, dtype=torch.uint8, device=DEV)  # NaN until written
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        self.state = torch.tensor([0, blocks, 0], dtype=torch.int64, device=DEV)
        self.ctx = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.latent_w, self.q_w = self.bf16(512), self.bf16(NOPE + 64)
        self.w_uk = self.bf16(HEADS, NOPE, 512) * NOPE ** -0.5
        self.inv = INV.to(DEV)

    def bf16(self, *shape):
        return torch.randn(shape, generator=self.gen, device=DEV).to(torch.bfloat16)

    def inputs(self, n):
        return self.bf16(n, 576), self.bf16(n, HEADS, NOPE + 64)

    def append(self, kv, q, new, slots_cap, first_position=0):
        """Blocks and slots for `new` tokens a request, the tokens into the cache; (q_out, slots, positions)."""
        slots, pos, start, _, _ = self.m.mla_block_table_extend(
            self.ctx, new, self.table, self.free, self.state, self.blocks, slots_cap, context_lens_out=self.ctx,
            free_state_out=self.state)
        pos = pos + first_position
        q_out = self.m.mla_kv_norm_rope_append(kv, self.latent_w, pos, self.inv, slots, self.pool, self.blocks, 64,
                                               self.stride, fmt=self.fmt, q=q, q_weight=self.q_w, rope_offset=NOPE)
        return q_out, slots, pos, start

    def decode_queries(self, q_out, q_len):
        q_nope = torch.einsum("nhd,hdl->nhl", q_out[..., :NOPE], self.w_uk)
        return (q_nope.view(self.batch, q_len, HEADS, 512).contiguous(),
                q_out[..., NOPE:].reshape(self.batch, q_len, HEADS, 64).contiguous())

    def window(self, q_out, q_len, sinks, window):
        qn, qr = self.decode_queries(q_out, q_len)
        lse = torch.empty((self.batch, q_len, HEADS), device=DEV)
        out, _ = self.m.mla_window_decode(qn, qr, self.pool, self.stride, self.blocks, self.table, self.ctx, SCALE,
                                          sinks, window, fmt=self.fmt, lse=lse)
        return out, lse, qn, qr

    def rows(self, b, positions):
        return rows64(self.pool, self.fmt, self.table[b], torch.as_tensor(positions, dtype=torch.int64, device=DEV))


def check_append(s, kv, q, q_out, slots, pos):
    """q_out and the cached bytes of the tokens that have a slot."""
    live = slots >= 0
    ref, size = heads64(q, s.q_w, pos, NOPE, True)
    assert_heads(q_out[live], ref[live], size[live])
    # the bytes that the quantised write gives for the normed, rotated bf16 rows
    # (their own roundings are checked where that operator is)
    x = kv.double()
    lat = x[:, :512] / torch.sqrt(x[:, :512].square().mean(-1, keepdim=True) + EPS) * s.latent_w.double()
    got = s.pool.view(-1, 64, ROW_BYTES[s.fmt])[slots[live] // 64, slots[live] % 64]
    key = got[:, -64:].view(torch.float8_e4m3fn).double()
    rot, mag = heads64(kv[:, None, 512:], None, pos, 0, True)
    rot, mag = rot[live, 0], mag[live, 0]
    # bf16 (2^-8) then e4m3 (2^-4 of the value, 2^-10 below its normal range)
    assert ((key - rot).abs() <= (2.0 ** -4 + 2.0 ** -7) * rot.abs() + 2.0 ** -10 + 2.0 ** -18 * mag).all()
    if s.fmt == 1:
        lat8 = got[:, :512].view(torch.float8_e4m3fn).double()
        assert ((lat8 - lat[live]).abs() <= (2.0 ** -4 + 2.0 ** -7) * lat[live].abs() + 2.0 ** -10).all()
    else:
        bits = u16(lat[live].to(torch.bfloat16))
        zero = np.zeros((bits.shape[0], 64), dtype=np.uint16)
        pool = np.zeros(-(-len(bits) // 64) * 64 * 352, dtype=np.uint8)
        O.kv_quantize_append(bits, zero, np.arange(len(bits), dtype=np.int64), pool, len(pool) // (64 * 352), 64,
                             64 * 352, 0)
        want = torch.from_numpy(pool.reshape(-1, 352)[:len(bits), :288]).to(DEV)
        # the kernel's float norm may round a bf16 value to the other neighbour, which can move a code or a
        # scale by one: bytes that differ stay rare (a tie within 2^-16 of a step, 800 bytes a row)
        assert (got[:, :288] != want).float().mean() <= 0.01


@pytest.mark.parametrize("fmt", [0, 1])
def test_prefill_then_window_steps(m, fmt):
    """Ragged prompts into an empty cache, then steps of two tokens that cross block and window edges."""
    batch, q_len, sinks, window = 5, 2, 4, 100
    s = Server(m, fmt, batch, 40, 5, 7 + fmt)
    table, free, state, ctx = s.table.tolist(), s.free.tolist(), s.state.tolist(), [0] * batch
    prompt = [1, 62, 126, 0, 190]
    for step, new in enumerate([prompt] + [[q_len] * batch] * 4):
        cap = sum(new) + (3 if step == 0 else 0)  # the prompts' call has room to spare
        kv, q = s.inputs(cap)
        q_out, slots, pos, start = s.append(kv, q, torch.tensor(new, dtype=torch.int32, device=DEV), cap)
        want = extend_loop(ctx, new, table, free, state, s.blocks, cap)
        for got, w in zip((slots, pos, start, s.ctx, s.state, s.table), want):
            assert got.tolist() == list(w)
        ctx, state, table = want[3], want[4], want[5]
        check_append(s, kv, q, q_out, slots, pos)
        if step == 0:
            continue
        out, lse, qn, qr = s.window(q_out, q_len, sinks, window)
        for b in range(batch):
            for i in range(q_len):
                seen = window_positions(ctx[b], q_len, i, sinks, window, 64 * len(table[b]))
                assert_attention(out[b, i], lse[b, i], *attend64(qn[b, i], qr[b, i], s.rows(b, seen)),
                                 what=f"step {step}, request {b}, token {i}")
    assert m.mla_device_fault() == 0


def test_shared_prefix_steps(m):
    """One request's prompt becomes the prefix of a batch whose requests then grow behind it."""
    prefix = 150
    base = Server(m, 0, 1, 64, 3, 11)
    kv, q = base.inputs(prefix)
    base.append(kv, q, torch.tensor([prefix], dtype=torch.int32, device=DEV), prefix)
    s = Server(m, 0, 6, 64, 2, 12)
    s.pool, s.latent_w, s.q_w, s.w_uk = base.pool, base.latent_w, base.q_w, base.w_uk
    s.free, s.state = base.free, base.state  # one pool, one ring
    for step, new in enumerate([[30, 64, 63, 1, 100, 7], [1] * 6, [1] * 6]):
        kv, q = s.inputs(sum(new))
        q_out, slots, pos, _ = s.append(kv, q, torch.tensor(new, dtype=torch.int32, device=DEV), sum(new), prefix)
        check_append(s, kv, q, q_out, slots, pos)
        if step == 0:
            continue
        qn, qr = s.decode_queries(q_out, 1)
        lse = torch.empty((6, 1, HEADS), device=DEV)
        out, _ = m.mla_prefix_decode(qn, qr, s.pool, s.stride, s.blocks, base.table[0], prefix, s.table, s.ctx, SCALE,
                                     128, lse=lse)
        for b in range(6):
            rows = torch.cat([base.rows(0, range(prefix)), s.rows(b, range(int(s.ctx[b])))])
            assert_attention(out[b, 0], lse[b, 0], *attend64(qn[b, 0], qr[b, 0], rows), what=f"request {b}")
    taken = torch.cat([base.table.flatten(), s.table.flatten()])
    taken = taken[taken >= 0].tolist()
    assert len(set(taken)) == len(taken) == int(s.state[0])  # no block was given twice
    assert m.mla_device_fault() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_captured_step_replays_like_the_eager_one(m, fmt):
    """The whole step in one graph: its lengths, tables and ring state advance on the device, and steps with
    fewer tokens than it was captured for leave the rest of the cache alone."""
    batch, q_len, sinks, window = 4, 2, 2, 70
    prompt = torch.tensor([0, 63, 64, 127], dtype=torch.int32, device=DEV)
    servers = []
    for _ in range(2):
        s = Server(m, fmt, batch, 32, 6, 21)
        s.append(*s.inputs(256), prompt, 256)
        servers.append(s)
    eager, s = servers
    assert torch.equal(eager.pool, s.pool) and torch.equal(eager.table, s.table)
    kv, q = s.inputs(batch * q_len)
    new = torch.zeros(batch, dtype=torch.int32, device=DEV)

    def step(x):
        q_out, slots, pos, start = x.append(kv, q, new, batch * q_len)
        return (*x.window(q_out, q_len, sinks, window)[:2], slots, pos, start)

    keep = [t.clone() for t in (s.table, s.ctx, s.state, s.pool)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # no new token: changes nothing
        step(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (s.table, s.ctx, s.state, s.pool)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    assert all(torch.equal(a, b) for a, b in zip(keep, (s.table, s.ctx, s.state, s.pool)))
    for i, lens in enumerate([[2, 2, 2, 2], [2, 2, 2, 2], [2, 0, 2, 1], [0, 0, 0, 0], [2, 2, 2, 2]]):
        new.copy_(torch.tensor(lens, dtype=torch.int32))
        a, b = s.inputs(batch * q_len)
        kv.copy_(a)
        q.copy_(b)
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for name, x, y in zip(("out", "lse", "slots", "positions", "starts"), got, want):
            assert torch.equal(x, y), (i, name)
        for name in ("table", "ctx", "state", "pool"):
            assert torch.equal(getattr(s, name), getattr(eager, name)), (i, name)
    assert m.mla_device_fault() == 0


def test_two_graphs_share_a_workspace_in_turn(m):
    """Captured calls of different shapes on one workspace: what one leaves in it does not reach the other."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    blocks = 80
    pool = torch.randint(0, 0x70, (blocks, 64 * 576), generator=g, device=DEV).to(torch.uint8)  # finite e4m3
    table = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32).view(2, 40)
    ctx = torch.tensor([2500, 900], dtype=torch.int32, device=DEV)
    qs = [torch.randn((2, n, HEADS, 576), generator=g, device=DEV).to(torch.bfloat16) for n in (1, 3)]
    args = [(q[..., :512].contiguous(), q[..., 512:].contiguous(), pool, 64 * 576, blocks) for q in qs]
    calls = [
        lambda **kw: m.mla_window_decode(*args[0], table, ctx, SCALE / 64, 2, 2000, fmt=1, **kw),
        lambda **kw: m.mla_prefix_decode(*args[1], table[0], 700, table, ctx, SCALE / 64, 2560, fmt=1, **kw),
    ]
    want = [c()[0].clone() for c in calls]
    need = max(m.mla_window_decode_workspace_size(2, 1, HEADS, 40, 2, 2000),
               m.mla_prefix_decode_workspace_size(2, 3, HEADS, 700, 40, 2560))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN where nothing was written
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for c, o in zip(calls, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c(out=o, workspace=ws)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i]), i
    assert m.mla_device_fault() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (48, 1), (48, 2), (64, 4)])
def test_many_calls_in_a_row(m, fmt, heads, q_len):
    """Calls queued without a pause give what each gives alone: the rows come from L2 and every ring of copies
    and tiles runs at its fastest."""
    g = torch.Generator(device=DEV)
    g.manual_seed(heads + q_len)
    batch, width = 20, 63
    rb = ROW_BYTES[fmt]
    pool = torch.randint(0, 0x70, (batch * width, 64 * rb), generator=g, device=DEV).to(torch.uint8)
    table = torch.randperm(batch * width, generator=g, device=DEV).to(torch.int32).view(batch, width)
    ctx = torch.randint(0, 4000, (batch,), generator=g, device=DEV).to(torch.int32)
    q = torch.randn((batch, q_len, heads, 576), generator=g, device=DEV).to(torch.bfloat16) / 64
    qn, qr = q[..., :512].contiguous(), q[..., 512:].contiguous()

    def call():
        return m.mla_window_decode(qn, qr, pool, 64 * rb, batch * width, table, ctx, SCALE, 7, 1500, fmt=fmt)[0]

    want = call()
    torch.cuda.synchronize()
    for _ in range(8):
        got = [call() for _ in range(24)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)
    assert m.mla_device_fault() == 0
