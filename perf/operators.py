"""Work around the paged latent cache, measured operator by operator.

Five operators of one serving step: block tables and slot maps from request
lengths (`extend`), norms and rotation of queries and keys (`norm_rope`), the
same pass writing the key into the paged cache (`append`), decode over a
sliding window with first tokens that stay visible (`window`), and decode of a
batch that shares a long prefix (`prefix`).  `run` computes each in its plain
form, or with `own` set calls the framework.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK, LATENT, ROPE, ROW = 64, 512, 64, 576
ROW_BYTES = {"nvfp4": 352, "fp8": 576}
SCALE = 1.0 / math.sqrt(192.0)
THETA, EPS = 10000.0, 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # every request of a running batch grows by the token it has just decoded: latency
        dict(name="extend_decode", op="extend", batch=128, ctx=140000, new=1, ragged=True),
        # 64 agents' turns of up to 6,000 tokens after a long prefix
        dict(name="extend_turn", op="extend", batch=64, ctx=140000, new=6000, ragged=True),
        # index queries (32 heads) and the index key of a decode batch
        dict(name="norm_rope_index", op="norm_rope", tokens=64, q_heads=32, k_heads=1, dim=128, offset=64, far=140000,
             interleaved=False),
        # one prefill turn: per-head queries and keys of 128 + 64 dims
        dict(name="norm_rope_turn", op="norm_rope", tokens=6000, q_heads=16, k_heads=16, dim=192, offset=128,
             far=1048576, interleaved=True),
        # one turn's latents into the 4-bit cache, its queries in the same pass
        dict(name="append_nvfp4_turn", op="append", fmt="nvfp4", tokens=6001, q_heads=16, far=140000,
             interleaved=True),
        # 64 sessions' turns into the FP8 cache, no queries
        dict(name="append_fp8_sessions", op="append", fmt="fp8", tokens=384000, q_heads=0, far=146000,
             interleaved=False),
        # one user's token: latency
        dict(name="window_one", op="window", fmt="nvfp4", batch=1, q_len=1, heads=16, ctx=140000, sinks=4, window=1000),
        # a tensor-parallel rank's batch with a wide window
        dict(name="window_rank", op="window", fmt="nvfp4", batch=32, q_len=1, heads=16, ctx=140000, sinks=64,
             window=8192),
        # draft tokens over an FP8 cache, ragged contexts, some shorter than the window
        dict(name="window_draft_fp8", op="window", fmt="fp8", batch=64, q_len=4, heads=16, ctx=5000, sinks=4,
             window=2047),
        # all 64 heads of a data-parallel rank
        dict(name="window_heads", op="window", fmt="nvfp4", batch=128, q_len=1, heads=64, ctx=16384, sinks=16,
             window=4096),
        # 32 agents on one 140,000-token prefix, each with up to 6,000 tokens of its own
        dict(name="prefix_agents", op="prefix", fmt="nvfp4", batch=32, q_len=1, heads=16, prefix=140000, ctx=6000),
        # a few samples of one prompt, all heads, two query tokens
        dict(name="prefix_samples_fp8", op="prefix", fmt="fp8", batch=8, q_len=2, heads=64, prefix=9001, ctx=500),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("extend", "norm_rope", "append", "window", "prefix"))
    fmt = rng.choice(("nvfp4", "fp8"))
    if op == "extend":
        batch = log(1, 2048)
        return dict(op=op, batch=batch, ctx=log(1, 140000), new=log(1, max(2, min(6000, 380000 // batch))),
                    ragged=rng.random() < 0.8)
    if op == "norm_rope":
        dim, offset = rng.choice(((64, 0), (128, 0), (128, 64), (192, 128), (256, 192)))
        return dict(op=op, tokens=log(1, 6000), q_heads=rng.choice((1, 8, 16, 32)), k_heads=rng.choice((0, 1, 8, 16)),
                    dim=dim, offset=offset, far=log(64, 1048576), interleaved=rng.random() < 0.5)
    if op == "append":
        return dict(op=op, fmt=fmt, tokens=log(1, 20000), q_heads=rng.choice((0, 16, 32)), far=log(64, 1048576),
                    interleaved=rng.random() < 0.5)
    if op == "window":
        heads, batch, q_len = rng.choice((16, 32, 48, 64)), log(1, 128), rng.choice((1, 1, 2, 4, 7))
        return dict(op=op, fmt=fmt, batch=batch, q_len=q_len, heads=heads, ctx=log(1, 16384),
                    sinks=rng.choice((0, 1, 4, 64, 100)), window=log(1, min(4096, 40000000 // (batch * q_len * heads))))
    batch, q_len, heads = log(2, 64), rng.choice((1, 1, 2, 3)), rng.choice((16, 32, 64))
    return dict(op=op, fmt=fmt, batch=batch, q_len=q_len, heads=heads,
                prefix=log(1, min(60000, 40000000 // (batch * q_len * heads))), ctx=log(1, 2000))


def lengths(case, key="ctx"):
    """Whole numbers up to case[key], the same for every seed: the batch's cached tokens."""
    n, top = case["batch"], case[key]
    if not case.get("ragged", True):
        return np.full(n, top, np.int64)
    x = (np.arange(n, dtype=np.int64) * 2654435761 + 40503 * (top + n)) % 1000003 / 1000003.0
    x = np.maximum(1, np.rint(top * (0.25 + 0.75 * x))).astype(np.int64)
    x[0] = top
    return x


def new_lengths(case):
    x = lengths(case, "new")
    if case["batch"] > 2:
        x[1] = 0  # a request that waits
    return x


def blocks(n):
    return -(-n // BLOCK)


def rows_read(case):
    """Cached rows that a decode cannot do without."""
    ctx = lengths(case)
    if case["op"] == "prefix":
        return case["prefix"] + int(ctx.sum())
    return int(np.minimum(ctx, case["sinks"] + case["window"] + case["q_len"] - 1).sum())


def work(case):
    op = case["op"]
    if op == "extend":
        total, need = int(new_lengths(case).sum()), int((blocks(lengths(case) + new_lengths(case)) - blocks(lengths(case))).sum())
        return {"bytes": total * 12 + need * 8 + case["batch"] * 20 + 48, "flops": 0}
    if op == "norm_rope":
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 5 * n}
    if op == "append":
        t = case["tokens"]
        n = t * case["q_heads"] * 192
        return {"bytes": 4 * n + t * (2 * ROW + 12 + ROW_BYTES[case["fmt"]]), "flops": 5 * n + 8 * t * ROW}
    cols = case["batch"] * case["q_len"] * case["heads"]
    ctx = lengths(case)
    if op == "window":
        seen = int(np.minimum(ctx, case["sinks"] + case["window"]).sum()) * case["q_len"] * case["heads"]
    else:
        seen = cols * case["prefix"] + int(ctx.sum()) * case["q_len"] * case["heads"]
    return {"bytes": rows_read(case) * ROW_BYTES[case["fmt"]] + cols * (2 * ROW + 2 * LATENT + 4),
            "flops": 2 * (ROW + LATENT) * seen}


# --------------------------------------------------------------------------- inputs
def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def make_pool(g, n_blocks, fmt):
    """A cache pool whose rows hold plausible latents: 4-bit codes under scales near 0.4, or e4m3 values."""
    if fmt == "fp8":
        return torch.randn((n_blocks, BLOCK, ROW), generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    pool = torch.randint(0, 256, (n_blocks, BLOCK, 352), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand((n_blocks, BLOCK, 32), generator=g, device=DEV) * 0.4 + 0.2
    pool[..., 256:288] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    pool[..., 288:] = torch.randn((n_blocks, BLOCK, ROPE), generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def make_tables(g, counts, extra=0):
    """Block tables of requests with `counts` blocks each, scattered over one pool; -1 behind a request's last."""
    total = int(counts.sum()) + extra
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    width = max(1, int(counts.max()))
    col = torch.arange(width, device=DEV)
    n = torch.from_numpy(counts).to(DEV)
    start = torch.cumsum(n, 0) - n
    at = (start[:, None] + col).clamp(max=max(0, total - 1))
    return torch.where(col < n[:, None], perm[at], -1).to(torch.int32), perm[total - extra:], total


def prepare(case, seed):
    g = generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "extend":
        ctx, new = lengths(case), new_lengths(case)
        have, want = blocks(ctx), blocks(ctx + new)
        spare = int((want - have).sum()) + 97
        table, free, total = make_tables(g, have, spare)
        width = max(1, int(want.max()))
        s["table"] = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1).contiguous()
        s["free"] = free.contiguous()
        head = spare // 3  # the ring has been round once: the first free block stands in its middle
        s["state"] = torch.tensor([head, head + spare, 0], dtype=torch.int64, device=DEV)
        s["pool_blocks"], s["slots"] = total, int(new.sum()) + 5  # a few entries of padding
        s["context"] = torch.from_numpy(ctx).to(DEV, torch.int32)
        s["grow"] = torch.from_numpy(new).to(DEV, torch.int32)
        return s
    s["inv_freq"] = THETA ** (-torch.arange(0, ROPE, 2, device=DEV, dtype=torch.float64) / ROPE)
    if op in ("norm_rope", "append"):
        t = case["tokens"]
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
    if op == "norm_rope":
        d = case["dim"]
        s["q"], s["k"] = normal(g, t, case["q_heads"], d, scale=2.0), normal(g, t, case["k_heads"], d, scale=0.5)
        s["wq"], s["wk"] = (normal(g, d, scale=0.2) + 1 for _ in range(2))
    elif op == "append":
        s["kv"] = normal(g, t, ROW, scale=1.5)
        s["w"] = normal(g, LATENT, scale=0.2) + 1
        s["q"] = normal(g, t, case["q_heads"], 192) if case["q_heads"] else None
        s["wq"] = normal(g, 192, scale=0.2) + 1
        n = blocks(t) + 1
        s["pool"] = make_pool(g, n, case["fmt"])
        s["slots"] = torch.randperm(n * BLOCK, generator=g, device=DEV)[:t].contiguous()
        s["slots"][::1000] = -1  # a padded entry now and then
    else:
        n = lengths(case)
        s["context"] = torch.from_numpy(n).to(DEV, torch.int32)
        p = blocks(case["prefix"]) if op == "prefix" else 0
        s["table"], s["prefix_table"], total = make_tables(g, blocks(n), p)
        s["prefix_table"] = s["prefix_table"].contiguous()
        s["pool"] = make_pool(g, total, case["fmt"])
        shape = (case["batch"], case["q_len"], case["heads"])
        s["q_nope"], s["q_rope"] = normal(g, *shape, LATENT), normal(g, *shape, ROPE)
        s["lse"] = torch.empty(shape, dtype=torch.float32, device=DEV)
        s["max_ctx"] = int(n.max())
    return s


# --------------------------------------------------------------------------- plain forms
def extend_plain(s):
    ctx, new, table = s["context"].long(), s["grow"].long(), s["table"]
    head, tail = s["state"][0], s["state"][1]
    ends = torch.cumsum(new, 0)
    start = torch.cat([ends.new_zeros(1), ends]).clamp(max=s["slots"])
    new = start[1:] - start[:-1]
    have, width = (ctx + BLOCK - 1) // BLOCK, table.shape[1]
    want = torch.minimum((ctx + new + BLOCK - 1) // BLOCK, torch.full_like(ctx, width))
    need = (want - have).clamp(min=0)
    before = torch.cumsum(need, 0) - need
    left = tail - head
    granted = torch.minimum((left - before).clamp(min=0), need)
    col = torch.arange(width, device=table.device)
    rank = before[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    got = fresh & (rank < left)
    ids = s["free"][(head + rank.clamp(min=0)) % s["free"].numel()]
    table = torch.where(got, ids, torch.where(fresh, torch.full_like(ids, -1), table))
    out_ctx = torch.minimum(ctx + new, torch.maximum(ctx, (have + granted) * BLOCK))
    t = torch.arange(s["slots"], device=table.device)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True)
    inside = r < ctx.numel()
    r = r.clamp(max=ctx.numel() - 1)
    pos = ctx[r] + t - start[r]
    held = inside & (pos < out_ctx[r])
    block = table[r, (pos // BLOCK).clamp(0, width - 1)].long()
    held = held & (block >= 0) & (block < s["pool_blocks"])
    slots = torch.where(held, block * BLOCK + pos % BLOCK, -1)
    positions = torch.where(inside, pos, -1).int()
    after = torch.stack([head + granted.sum(), tail, (need - granted).sum()])
    return dict(slots=slots, positions=positions, start=start.int(), context=out_ctx.int(), state=after, table=table)


def normed(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def rotated(x, positions, inv_freq, interleaved):
    """x float32 [tokens, heads, 64] by the angles of its positions (far ones need 64 bits)."""
    a = positions.double()[:, None] * inv_freq
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    if interleaved:
        x, y = x[..., 0::2], x[..., 1::2]
        return torch.stack([x * c - y * s, y * c + x * s], -1).flatten(-2)
    x, y = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([x * c - y * s, y * c + x * s], -1)


def head_plain(x, w, positions, inv_freq, offset, interleaved):
    x = normed(x, w)
    turned = rotated(x[..., offset:offset + ROPE], positions, inv_freq, interleaved)
    return torch.cat([x[..., :offset], turned, x[..., offset + ROPE:]], -1).to(torch.bfloat16)


def e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def e2m1(x):
    """The nearest e2m1 value, ties to the even code."""
    a = x.abs()
    up = (a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0)
    step = (0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0)
    return torch.copysign(sum(u * d for u, d in zip(up, step)), x)


def pool_values(pool, fmt):
    """What a pool's bytes stand for: e2m1 codes, their scales and the rope values, each held in e4m3."""
    if fmt == "fp8":
        return dict(row=pool.view(torch.float8_e4m3fn))
    both = torch.tensor([v * f for f in (1.0, -1.0) for v in E2M1], device=pool.device)
    code = torch.arange(256, device=pool.device)
    pair = torch.stack([both[code & 15], both[code >> 4]], -1).to(torch.float8_e4m3fn).view(torch.int16).flatten()
    n = pool.shape[0]
    latent = pair.index_select(0, pool[..., :256].int().flatten()).view(torch.float8_e4m3fn)
    return dict(latent=latent.view(n, BLOCK, LATENT), scale=pool[..., 256:288].view(torch.float8_e4m3fn),
                rope=pool[..., 288:].view(torch.float8_e4m3fn))


def append_plain(s):
    latent = normed(s["kv"][:, :LATENT], s["w"]).to(torch.bfloat16).float()
    rope = rotated(s["kv"][:, None, LATENT:].float(), s["positions"], s["inv_freq"], s["interleaved"])
    rope = e4m3(rope[:, 0].to(torch.bfloat16).float())
    out = {k: v.clone().view(torch.uint8) for k, v in pool_values(s["pool"], s["fmt"]).items()}
    keep = s["slots"] >= 0
    at = s["slots"].clamp(min=0)

    def put(name, rows):
        rows, to = rows.view(torch.uint8), out[name].view(-1, rows.shape[-1])
        # a skipped token's slot is taken from a kept one, whose row it writes again
        first = keep.to(torch.uint8).argmax()
        source = torch.where(keep, torch.arange(keep.numel(), device=keep.device), first)
        to.index_copy_(0, at[source], rows[source])

    if s["fmt"] == "fp8":
        put("row", torch.cat([e4m3(latent).view(torch.uint8), rope.view(torch.uint8)], -1).view(torch.float8_e4m3fn))
    else:
        x = latent.view(-1, 32, 16)
        scale = e4m3(x.abs().amax(-1) / 6.0)
        sf = scale.float()[..., None]
        codes = torch.where(sf > 0, e2m1(x / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(x))
        put("latent", codes.flatten(-2).to(torch.float8_e4m3fn))
        put("scale", scale)
        put("rope", rope)
    out = {k: v.view(torch.float8_e4m3fn) for k, v in out.items()}
    if s["q"] is not None:
        out["q"] = head_plain(s["q"], s["wq"], s["positions"], s["inv_freq"], 128, s["interleaved"])
    return out


def gathered(pool, fmt, table, positions):
    """The cached rows of `positions` [..., n] through `table` [..., blocks], as float32 [..., n, 576]."""
    block = torch.gather(table.long(), -1, (positions // BLOCK).clamp(0, table.shape[-1] - 1)).clamp(min=0)
    raw = pool[block, positions % BLOCK]
    if fmt == "fp8":
        return raw.view(torch.float8_e4m3fn).float()
    value = torch.tensor([v * f for f in (1.0, -1.0) for v in E2M1], device=pool.device)
    codes = torch.stack([raw[..., :256] & 15, raw[..., :256] >> 4], -1).flatten(-2).int()
    scale = raw[..., 256:288].view(torch.float8_e4m3fn).float()
    latent = value.index_select(0, codes.flatten()).view(*raw.shape[:-1], 32, 16) * scale[..., None]
    return torch.cat([latent.flatten(-2), raw[..., 288:].view(torch.float8_e4m3fn).float()], -1)


def blend(z, value):
    """(softmax(z) . value, log-sum-exp) over z's last axis; a row of -inf gives zeros and -inf."""
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, value) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (m + torch.log(total))[..., 0]


def window_plain(s):
    b, q, h = s["lse"].shape
    ctx = s["context"].long()[:, None]
    sinks = s["sinks"]
    j = torch.arange(sinks + min(s["window"] + q - 1, s["max_ctx"]), device=ctx.device)
    first = (ctx - q - s["window"] + 1).clamp(min=sinks)
    pos = torch.where(j < sinks, j, first + j - sinks)
    rows = gathered(s["pool"], s["fmt"], s["table"], pos)
    me = ctx - q + torch.arange(q, device=ctx.device)
    seen = (pos[:, None] <= me[..., None]) & ((pos[:, None] < sinks) | (pos[:, None] > me[..., None] - s["window"]))
    query = torch.cat([s["q_nope"], s["q_rope"]], -1).float().view(b, q * h, ROW)
    z = torch.matmul(query, rows.transpose(1, 2)).view(b, q, h, -1) * SCALE
    z = z.masked_fill(~seen[:, :, None], -math.inf).view(b, q * h, -1)
    out, lse = blend(z, rows[..., :LATENT])
    return out.view(b, q, h, LATENT).to(torch.bfloat16), lse.view(b, q, h)


def prefix_plain(s):
    b, q, h = s["lse"].shape
    ctx = s["context"].long()[:, None]
    query = torch.cat([s["q_nope"], s["q_rope"]], -1).float()
    shared = gathered(s["pool"], s["fmt"], s["prefix_table"], torch.arange(s["prefix"], device=ctx.device))
    z0 = torch.matmul(query.view(b * q * h, ROW), shared.t()) * SCALE
    out0, lse0 = blend(z0, shared[:, :LATENT])
    pos = torch.arange(s["max_ctx"], device=ctx.device).expand(b, -1)
    rows = gathered(s["pool"], s["fmt"], s["table"], pos)
    me = ctx - q + torch.arange(q, device=ctx.device)
    z1 = torch.matmul(query.view(b, q * h, ROW), rows.transpose(1, 2)).view(b, q, h, -1) * SCALE
    z1 = z1.masked_fill(~(pos[:, None] <= me[..., None])[:, :, None], -math.inf).view(b, q * h, -1)
    out1, lse1 = blend(z1, rows[..., :LATENT])
    out0, lse0, lse1 = out0.view(b, q * h, LATENT), lse0.view(b, q * h), lse1.view(b, q * h)
    m = torch.maximum(lse0, lse1)
    w0, w1 = torch.exp(lse0 - m), torch.exp(lse1 - m)
    out = (out0 * w0[..., None] + out1 * w1[..., None]) / (w0 + w1)[..., None]
    return out.view(b, q, h, LATENT).to(torch.bfloat16), (m + torch.log(w0 + w1)).view(b, q, h)


# --------------------------------------------------------------------------- one pass
def run_own(s):
    import sparse_mla_decode_kv_gb300 as mla

    op = s["op"]
    if op == "extend":
        slots, positions, start, context, state = mla.mla_block_table_extend(
            s["context"], s["grow"], s["table"], s["free"], s["state"], s["pool_blocks"], s["slots"])
        return dict(slots=slots, positions=positions, start=start, context=context, state=state, table=s["table"])
    if op == "norm_rope":
        return mla.mla_qk_norm_rope(s["q"], s["k"] if s["k_heads"] else None, s["positions"], s["inv_freq"],
                                    q_weight=s["wq"], k_weight=s["wk"], eps=EPS, rope_offset=s["offset"],
                                    interleaved=s["interleaved"])
    fmt = mla.MLA_KV_NVFP4 if s["fmt"] == "nvfp4" else mla.MLA_KV_FP8
    stride = BLOCK * ROW_BYTES[s["fmt"]]
    if op == "append":
        q = mla.mla_kv_norm_rope_append(s["kv"], s["w"], s["positions"], s["inv_freq"], s["slots"], s["pool"],
                                        s["pool"].shape[0], BLOCK, stride, fmt, eps=EPS,
                                        interleaved=s["interleaved"], q=s["q"], q_weight=s["wq"], rope_offset=128)
        out = pool_values(s["pool"], s["fmt"])
        return out if q is None else dict(out, q=q)
    if op == "window":
        return mla.mla_window_decode(s["q_nope"], s["q_rope"], s["pool"], stride, s["pool"].shape[0], s["table"],
                                     s["context"], SCALE, s["sinks"], s["window"], fmt=fmt, lse=s["lse"])
    return mla.mla_prefix_decode(s["q_nope"], s["q_rope"], s["pool"], stride, s["pool"].shape[0], s["prefix_table"],
                                 s["prefix"], s["table"], s["context"], SCALE, s["max_ctx"], fmt=fmt, lse=s["lse"])


def run(s):
    if own:
        return run_own(s)
    op = s["op"]
    if op == "extend":
        return extend_plain(s)
    if op == "norm_rope":
        q, k = (head_plain(x, w, s["positions"], s["inv_freq"], s["offset"], s["interleaved"]) if x.shape[1] else None
                for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
        return q, k
    return {"append": append_plain, "window": window_plain, "prefix": prefix_plain}[op](s)


# --------------------------------------------------------------------------- in 64 bits
def exact_extend(s):
    ctx, new = s["context"].tolist(), s["grow"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
    head, tail = s["state"].tolist()[:2]
    slots, positions = np.full(s["slots"], -1, np.int64), np.full(s["slots"], -1, np.int32)
    start, grown, at, missing = [0], [], 0, 0
    for b in range(len(ctx)):
        n = min(new[b], s["slots"] - at)
        room = blocks(ctx[b])
        for c in range(room, min(blocks(ctx[b] + n), table.shape[1])):
            if head < tail:
                table[b, c], head, room = free[head % len(free)], head + 1, c + 1
            else:
                table[b, c], missing = -1, missing + 1
        end = min(ctx[b] + n, max(ctx[b], room * BLOCK))
        pos = np.arange(ctx[b], ctx[b] + n)
        ids = table[b, np.minimum(pos // BLOCK, table.shape[1] - 1)].astype(np.int64)
        good = (pos < end) & (ids >= 0) & (ids < s["pool_blocks"])
        slots[at:at + n] = np.where(good, ids * BLOCK + pos % BLOCK, -1)
        positions[at:at + n] = pos
        at += n
        start.append(at)
        grown.append(end)
    return dict(slots=slots, positions=positions, start=np.array(start, np.int32), context=np.array(grown, np.int32),
                state=np.array([head, tail, missing], np.int64), table=table)


def exact_heads(x, w, s, offset):
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    return exact_turn(x, s, offset)


def exact_turn(x, s, offset):
    """Each pair as a complex number times e^(i angle)."""
    x = x.clone()
    part = x[..., offset:offset + ROPE]
    pair = part.unflatten(-1, (ROPE // 2, 2)) if s["interleaved"] else part.unflatten(-1, (2, ROPE // 2)).transpose(-1, -2)
    angle = s["positions"].double().view(-1, *([1] * (x.dim() - 1))) * s["inv_freq"]
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    pair = torch.view_as_real(z)
    x[..., offset:offset + ROPE] = (pair if s["interleaved"] else pair.transpose(-1, -2)).flatten(-2)
    return x


def exact_append(s):
    kv = s["kv"].double()
    latent = kv[:, :LATENT] / torch.sqrt(kv[:, :LATENT].square().mean(-1, keepdim=True) + EPS) * s["w"].double()
    rope = exact_turn(kv[:, LATENT:], s, 0)
    # the cache holds what bf16 rows would be stored as
    latent, rope = latent.to(torch.bfloat16).double(), rope.to(torch.bfloat16).double()
    grid8 = torch.arange(127, device=kv.device, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    grid4 = torch.tensor(E2M1, device=kv.device, dtype=torch.float64)

    def nearest(x, grid):
        a = x.abs().contiguous()
        hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
        lo = hi - 1
        below, above = a - grid[lo], grid[hi] - a
        at = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
        return torch.copysign(grid[at], x)

    keep = s["slots"] >= 0
    at = s["slots"][keep]
    out = {k: v.float().double() for k, v in pool_values(s["pool"], s["fmt"]).items()}
    if s["fmt"] == "fp8":
        out["row"].view(-1, ROW)[at] = nearest(torch.cat([latent, rope], -1), grid8)[keep]
    else:
        g = latent.unflatten(-1, (32, 16))
        scale = nearest(g.abs().amax(-1) / 6, grid8)
        codes = nearest(g / scale.clamp(min=1e-30)[..., None], grid4) * (scale > 0)[..., None]
        out["latent"].view(-1, LATENT)[at] = codes.flatten(-2)[keep]
        out["scale"].view(-1, 32)[at] = scale[keep]
        out["rope"].view(-1, ROPE)[at] = nearest(rope, grid8)[keep]
    if s["q"] is not None:
        out["q"] = exact_heads(s["q"], s["wq"], s, 128)
    return out


def exact_rows(s, table, n):
    """The first n rows of one request's (or the prefix's) cache in float64 [n, 576]."""
    t = torch.arange(n, device=DEV)
    raw = s["pool"].view(-1, s["pool"].shape[-1])[table.long()[t // BLOCK] * BLOCK + t % BLOCK]
    if s["fmt"] == "fp8":
        return raw.view(torch.float8_e4m3fn).double()
    nibble = torch.stack([raw[:, :256] % 16, raw[:, :256] // 16], -1).flatten(1).long()
    mag = torch.tensor(E2M1, device=DEV, dtype=torch.float64)[nibble % 8] * (1 - 2 * (nibble // 8))
    scale = raw[:, 256:288].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return torch.cat([mag * scale, raw[:, 288:].view(torch.float8_e4m3fn).double()], 1)


def exact_decode(s):
    b, q, h = s["lse"].shape
    out = torch.zeros((b, q, h, LATENT), dtype=torch.float64, device=DEV)
    lse = torch.full((b, q, h), -math.inf, dtype=torch.float64, device=DEV)
    shared = exact_rows(s, s["prefix_table"], s["prefix"]) if s["op"] == "prefix" else None
    for r, n in enumerate(s["context"].tolist()):
        rows = exact_rows(s, s["table"][r], n)
        for i in range(q):
            me = n - q + i
            t = torch.arange(n, device=DEV)
            see = t <= me
            if s["op"] == "window":
                see &= (t < s["sinks"]) | (t > me - s["window"])
            seen = rows[see] if shared is None else torch.cat([shared, rows[see]])
            if not seen.shape[0]:
                continue
            z = torch.cat([s["q_nope"][r, i], s["q_rope"][r, i]], -1).double() @ seen.t() * SCALE
            lse[r, i] = torch.logsumexp(z, -1)
            out[r, i] = torch.softmax(z, -1) @ seen[:, :LATENT]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "extend":
        return exact_extend(s)
    if op == "norm_rope":
        return (exact_heads(s["q"], s["wq"], s, s["offset"]),
                exact_heads(s["k"], s["wk"], s, s["offset"]) if case["k_heads"] else None)
    return exact_append(s) if op == "append" else exact_decode(s)
