"""Plain float64 forms for the tests of the operators around the paged cache
(not collected as tests): dequantised rows, attention over an explicit set of
rows, block tables by a loop."""
import math

import torch

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
ROW_BYTES = (352, 576)
SCALE = 1.0 / math.sqrt(192.0)


def random_pool(gen, n_blocks, fmt, stride=None, device="cuda"):
    """(pool uint8 [n_blocks, stride], stride): rows of finite values, the bytes between blocks e4m3 NaN."""
    rb = ROW_BYTES[fmt]
    stride = stride or 64 * rb
    pool = torch.full((n_blocks, stride), 0x7F, dtype=torch.uint8, device=device)
    rows = torch.empty((n_blocks, 64, rb), dtype=torch.uint8, device=device)

    def e4m3(*shape):
        return torch.randn(shape, generator=gen, device=device).to(torch.float8_e4m3fn).view(torch.uint8)

    if fmt == 1:
        rows[:] = e4m3(n_blocks, 64, 576)
    else:
        rows[..., :256] = torch.randint(0, 256, (n_blocks, 64, 256), generator=gen, device=device).to(torch.uint8)
        rows[..., 256:288] = (torch.rand((n_blocks, 64, 32), generator=gen, device=device) * 0.4 + 0.2).to(
            torch.float8_e4m3fn).view(torch.uint8)
        rows[..., 288:] = e4m3(n_blocks, 64, 64)
    pool[:, :64 * rb] = rows.view(n_blocks, -1)
    return pool, stride


def rows64(pool, fmt, table_row, positions):
    """Dequantised rows float64 [n, 576] of one table's positions (all of them cached)."""
    rb = ROW_BYTES[fmt]
    p = positions.long()
    raw = pool[:, :64 * rb].reshape(-1, 64, rb)[table_row.long()[p // 64], p % 64]
    if fmt == 1:
        return raw.view(torch.float8_e4m3fn).double()
    codes = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], -1).flatten(1).long()
    scale = raw[:, 256:288].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return torch.cat([E2M1.to(pool.device)[codes] * scale, raw[:, 288:].view(torch.float8_e4m3fn).double()], 1)


def attend64(q_nope, q_rope, rows, scale=SCALE):
    """(out, lse, softmax . |V|) of queries [H, 512], [H, 64] over rows [n, 576]; zeros and -inf for n = 0."""
    h = q_nope.shape[0]
    if rows.shape[0] == 0:
        z = torch.zeros((h, 512), dtype=torch.float64, device=rows.device)
        return z, torch.full((h,), -math.inf, dtype=torch.float64, device=rows.device), z
    z = torch.cat([q_nope, q_rope], -1).double() @ rows.t() * scale
    p = torch.softmax(z, -1)
    return p @ rows[:, :512], torch.logsumexp(z, -1), p @ rows[:, :512].abs()


def window_positions(ctx, q_len, i, sinks, window, held):
    """Positions that query token i sees: those up to its own among the first `sinks` and the last `window`."""
    me = ctx - q_len + i
    return [t for t in range(min(me + 1, held)) if t < sinks or t > me - window]


# One rounding is off by at most half a step: bf16 output 2^-8 of the value.  P
# and a slice's partial output are rounded to f16, 2^-11 each of the weighted
# magnitudes A = softmax . |V|.  A score's float accumulation over 576 products
# is off by at most 576 x 2^-24 x sum |q k| scale < 2^-10 for |q|, |k| ~ 1 (sum
# |q k| scale < 28), which moves the output by at most twice that share of A and
# the LSE by it.  exp2 / log2 approximations are 2^-21 and lost in it.
def out_tolerance(ref, a):
    return 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -9) * a + 1e-30


LSE_TOL = 2.0 ** -10


def assert_attention(out, lse, ref, ref_lse, a, what=""):
    err = (out.double() - ref).abs()
    over = (err - out_tolerance(ref, a)).max().item()
    assert over <= 0, f"{what}: out {over:.3e} past its tolerance (largest error {err.max().item():.3e})"
    inf = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), inf), f"{what}: -inf pattern of lse differs"
    if (~inf).any():
        d = (lse.double() - ref_lse)[~inf].abs().max().item()
        assert d <= LSE_TOL, f"{what}: lse off by {d:.3e}"


def extend_loop(ctx, new, table, free, state, pool_blocks, n_slots):
    """mla_block_table_extend one token at a time."""
    ctx, new, table = list(ctx), list(new), [list(r) for r in table]
    head, tail = state[0], state[1]
    width = len(table[0]) if table else 0
    left = max(0, min(tail - head, len(free)))
    slots, positions, start, out, taken, short = [], [], [0], [], 0, 0
    for b in range(len(ctx)):
        n = min(max(0, new[b]), n_slots - start[-1])
        c = max(0, ctx[b])
        have = -(-c // 64)
        room = have
        for col in range(have, min(-(-(c + n) // 64), width)):
            if taken < left:
                table[b][col] = free[(head + taken) % len(free)]
                taken, room = taken + 1, col + 1
            else:
                table[b][col], short = -1, short + 1
        end = min(c + n, max(c, min(room, width) * 64))
        for pos in range(c, c + n):
            block = table[b][pos // 64] if pos < end and pos // 64 < width else -1
            slots.append(block * 64 + pos % 64 if 0 <= block < pool_blocks else -1)
            positions.append(pos)
        start.append(start[-1] + n)
        out.append(end)
    pad = n_slots - start[-1]
    return slots + [-1] * pad, positions + [-1] * pad, start, out, [head + taken, tail, short], table
