"""Work around the attention of a layer, measured operator by operator.

Three operators that stand before and beside the cached decode: attention over
whole prompts packed one behind another (`attend`), the residual's addition and
norm with an output in 8 bits (`norm`), and matrix products of a few tokens with
weights in 4 bits (`matvec`).  `run` computes each in its plain form, or with
`own` set calls the framework.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # three requests' first few words, small heads: latency
        dict(name="attend_words", op="attend", batch=3, q=17, kv=17, ragged=True, heads=8, kv_heads=8, dk=64, dv=64,
             causal=True),
        # one agent's first turn on a tensor-parallel rank
        dict(name="attend_turn", op="attend", batch=1, q=6000, kv=6000, ragged=False, heads=16, kv_heads=16, dk=192,
             dv=128, causal=True),
        # a chunk of a long prompt, behind the tokens before it
        dict(name="attend_chunk", op="attend", batch=1, q=2048, kv=32768, ragged=False, heads=16, kv_heads=16, dk=192,
             dv=128, causal=True),
        # prompts of different lengths in one batch, grouped heads
        dict(name="attend_packed", op="attend", batch=16, q=1500, kv=1500, ragged=True, heads=32, kv_heads=4, dk=128,
             dv=128, causal=True),
        # one new token for each of a batch of requests, grouped heads
        dict(name="attend_tokens", op="attend", batch=32, q=1, kv=8192, ragged=True, heads=64, kv_heads=8, dk=128,
             dv=128, causal=True),
        # one user's token: latency
        dict(name="norm_token", op="norm", tokens=1, dim=6144, group=128, residual="bf16"),
        # rows of an odd width and number, a float residual, one scale a row
        dict(name="norm_odd", op="norm", tokens=1001, dim=1544, group=0, residual="f32"),
        # one prefill turn of four agents
        dict(name="norm_turn", op="norm", tokens=24000, dim=6144, group=128, residual="bf16"),
        # a decode batch's queries, each head's into the latent's 512 dims
        dict(name="matvec_heads", op="matvec", tokens=32, groups=16, n=512, k=128, x="bf16", out="bf16"),
        # one user's token through a wide projection, from the norm's 8 bits
        dict(name="matvec_token", op="matvec", tokens=1, groups=1, n=12288, k=6144, x="e4m3", out="bf16"),
        # four draft tokens, an odd number of outputs in float
        dict(name="matvec_drafts", op="matvec", tokens=4, groups=1, n=24583, k=6144, x="bf16", out="f32"),
        # a batch's tokens through the projection back, from 8 bits
        dict(name="matvec_batch", op="matvec", tokens=32, groups=1, n=6144, k=12288, x="e4m3", out="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("attend", "norm", "matvec"))
    if op == "attend":
        dk, dv = rng.choice(((64, 64), (128, 128), (192, 128), (96, 80)))
        kv_heads, group = rng.choice((1, 2, 4, 8, 16)), rng.choice((1, 1, 2, 4, 7, 8))
        heads, batch = kv_heads * group, log(1, 64)
        kv = log(1, min(20000, 400000000 // (batch * heads)))
        q = min(kv, log(1, max(1, min(kv, 400000000 // (batch * heads * kv)))))
        return dict(op=op, batch=batch, q=q, kv=kv, ragged=rng.random() < 0.8, heads=heads, kv_heads=kv_heads, dk=dk,
                    dv=dv, causal=rng.random() < 0.8)
    if op == "norm":
        return dict(op=op, tokens=log(1, 8000), dim=8 * log(8, 1024), group=rng.choice((0, 128, 128)),
                    residual=rng.choice(("bf16", "bf16", "f32", "none")))
    groups = rng.choice((1, 1, 1, 8, 16, 64))
    k = 32 * log(1, 512 if groups == 1 else 32)
    return dict(op=op, tokens=log(1, 64), groups=groups, n=log(1, min(16384, 100000000 // (groups * k))), k=k,
                x=rng.choice(("bf16", "e4m3")), out=rng.choice(("bf16", "f32")))


def lengths(case, key):
    """Whole numbers from 1 to case[key], the same for every seed: the batch's query or key tokens."""
    n, top = case["batch"], case[key]
    if not case["ragged"]:
        return np.full(n, top, np.int64)
    x = (np.arange(n, dtype=np.int64) * 2654435761 + 40503 * (top + n)) % 1000003 / 1000003.0
    x = np.maximum(1, np.rint(top * (0.1 + 0.9 * x))).astype(np.int64)
    x[0] = top
    return x


def both_lengths(case):
    """(query tokens, key tokens) of each sequence; a sequence has at least as many keys as queries."""
    kv = lengths(case, "kv")
    return np.minimum(lengths(case, "q"), kv), kv


def scale_count(case):
    """Scales of one row of 8-bit values."""
    return 1 if case.get("group", 128) == 0 else -(-case.get("dim", case.get("k")) // 128)


def work(case):
    op = case["op"]
    if op == "attend":
        nq, nk = both_lengths(case)
        h, hk, dk, dv = case["heads"], case["kv_heads"], case["dk"], case["dv"]
        seen = int((nq * nk - (nq * (nq - 1) // 2 if case["causal"] else 0)).sum()) * h
        return {"bytes": 2 * int(nq.sum()) * h * (dk + dv) + 2 * int(nk.sum()) * hk * (dk + dv) + 4 * int(nq.sum()) * h,
                "flops": 2 * (dk + dv) * seen}
    if op == "norm":
        n = case["tokens"] * case["dim"]
        r = {"bf16": 4, "f32": 8, "none": 0}[case["residual"]]
        return {"bytes": n * (2 + 1 + r) + 2 * case["dim"] + 4 * case["tokens"] * scale_count(case), "flops": 6 * n}
    t, g, n, k = (case[x] for x in ("tokens", "groups", "n", "k"))
    x = t * g * k * (2 if case["x"] == "bf16" else 1) + (0 if case["x"] == "bf16" else 4 * t * g * scale_count(case))
    return {"bytes": g * n * k * 9 // 16 + x + t * g * n * (2 if case["out"] == "bf16" else 4) + 4 * g,
            "flops": 2 * t * g * n * k}


# --------------------------------------------------------------------------- inputs
def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def starts(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)


def prepare(case, seed):
    g = generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "attend":
        nq, nk = both_lengths(case)
        s["q_start"], s["kv_start"] = starts(nq), starts(nk)
        s["max_q"], s["max_kv"] = int(nq.max()), int(nk.max())
        # keys and values of a token lie side by side, as the projection that makes them writes them
        dk, dv = case["dk"], case["dv"]
        s["queries"] = normal(g, int(nq.sum()), case["heads"], dk)
        kv = normal(g, int(nk.sum()), case["kv_heads"], dk + dv)
        s["keys"], s["values"] = kv[..., :dk], kv[..., dk:]
        s["scale"] = 2.0 / math.sqrt(dk)
    elif op == "norm":
        t, d = case["tokens"], case["dim"]
        s["x_in"] = normal(g, t, d, scale=0.7)
        s["res"] = None
        if case["residual"] != "none":
            # a few dims of a residual stream are far larger than the others
            r = torch.randn((t, d), generator=g, device=DEV) * 3.0
            r[:, :: max(1, d // 3)] *= 40.0
            s["res"] = r if case["residual"] == "f32" else r.to(torch.bfloat16)
        s["w"] = normal(g, d, scale=0.2) + 1
    else:
        t, n_g, n, k = (case[x] for x in ("tokens", "groups", "n", "k"))
        s["codes"] = torch.randint(0, 256, (n_g, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        u = torch.rand((n_g, n, k // 16), generator=g, device=DEV) * 200 + 20
        s["scales"] = u.to(torch.float8_e4m3fn)
        s["weight_scale"] = (torch.rand(n_g, generator=g, device=DEV) + 0.5) * 1e-4
        if case["x"] == "bf16":
            # a head's first k values of k + 64, as the rotation leaves them
            s["x_in"] = normal(g, t, n_g, k + 64)[..., :k]
            s["x_scales"] = None
        else:
            s["x_in"] = (torch.randn((t, n_g, k), generator=g, device=DEV) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["x_scales"] = torch.rand((t, n_g, scale_count(case)), generator=g, device=DEV) * 0.01 + 0.001
    return s


# --------------------------------------------------------------------------- plain forms
def attend_plain(s):
    nq, nk = s["q_start"][1:] - s["q_start"][:-1], s["kv_start"][1:] - s["kv_start"][:-1]
    i, j = (torch.arange(s[m], device=DEV) for m in ("max_q", "max_kv"))
    b, hk, dk, dv = s["batch"], s["kv_heads"], s["dk"], s["dv"]
    group = s["heads"] // hk
    at_q = (s["q_start"][:-1, None] + i).clamp(max=s["queries"].shape[0] - 1)
    at_k = (s["kv_start"][:-1, None] + j).clamp(max=s["keys"].shape[0] - 1)
    q = s["queries"][at_q].float().view(b, s["max_q"], hk, group, dk).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, dk)
    k, v = (s[m][at_k].float().permute(0, 2, 1, 3) for m in ("keys", "values"))
    last = (nk - nq)[:, None] + i if s["causal"] else (nk[:, None] - 1).expand(b, s["max_q"])
    seen = (j <= last[..., None]) & (j < nk[:, None, None])
    z = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hk, s["max_q"], group, -1)
    z = z.masked_fill_(~seen[:, None, :, None], -math.inf).view(b, hk, s["max_q"] * group, -1)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total))[..., 0]
    out = out.view(b, hk, s["max_q"], group, dv).permute(0, 2, 1, 3, 4).reshape(b, s["max_q"], s["heads"], dv)
    lse = lse.view(b, hk, s["max_q"], group).permute(0, 2, 1, 3).reshape(b, s["max_q"], s["heads"])
    t = torch.arange(s["queries"].shape[0], device=DEV)
    r = torch.searchsorted(s["q_start"][1:].long().contiguous(), t, right=True)
    return out[r, t - s["q_start"][r]].to(torch.bfloat16), lse[r, t - s["q_start"][r]]


def norm_plain(s):
    x = s["x_in"].float()
    h = x if s["res"] is None else x + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
    groups, d = scale_count(s), s["dim"]
    width = d if s["group"] == 0 else 128
    parts = torch.nn.functional.pad(y, (0, groups * width - d)).view(-1, groups, width)
    scales = parts.abs().amax(-1) / 448.0
    codes = parts / torch.where(scales > 0, scales, torch.ones_like(scales))[..., None]
    codes = codes.flatten(1)[:, :d].clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, scales, None if s["res"] is None else h.to(s["res"].dtype)


def matvec_plain(s):
    t, g, n, k = (s[x] for x in ("tokens", "groups", "n", "k"))
    x = s["x_in"].float()
    if s["x_scales"] is not None:
        x = x * s["x_scales"].repeat_interleave(128, -1)[..., :k]
    value = torch.tensor([v * f for f in (1.0, -1.0) for v in E2M1], device=DEV)
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).int().flatten()
    w = value.index_select(0, codes).view(g, n, k // 16, 16) * s["scales"].float()[..., None]
    y = torch.matmul(x.transpose(0, 1), w.view(g, n, k).transpose(1, 2)) * s["weight_scale"][:, None, None]
    return y.transpose(0, 1).to(torch.bfloat16 if s["out"] == "bf16" else torch.float32).contiguous()


# --------------------------------------------------------------------------- one pass
def run_own(s):
    import sparse_mla_decode_kv_gb300 as mla

    if s["op"] == "attend":
        lse = torch.empty(s["queries"].shape[:2], dtype=torch.float32, device=DEV)
        return mla.mla_prompt_attention(s["queries"], s["keys"], s["values"], s["q_start"], s["kv_start"], s["scale"],
                                        causal=s["causal"], lse=lse)
    if s["op"] == "norm":
        return mla.mla_add_norm_quant(s["x_in"], s["w"], residual=s["res"], eps=EPS, group=s["group"])
    return mla.mla_fp4_matvec(s["x_in"], s["codes"], s["scales"], s["weight_scale"], x_scales=s["x_scales"],
                              out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)


def run(s):
    if own:
        return run_own(s)
    return {"attend": attend_plain, "norm": norm_plain, "matvec": matvec_plain}[s["op"]](s)


# --------------------------------------------------------------------------- in 64 bits
def exact_attend(s):
    q_start, kv_start = s["q_start"].tolist(), s["kv_start"].tolist()
    total, heads, dv = s["queries"].shape[0], s["heads"], s["dv"]
    out = torch.zeros((total, heads, dv), dtype=torch.float64, device=DEV)
    lse = torch.full((total, heads), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(s["batch"]):
        q0, q1, k0, k1 = q_start[r], q_start[r + 1], kv_start[r], kv_start[r + 1]
        ahead = (k1 - k0) - (q1 - q0)
        hidden = torch.ones((q1 - q0, k1 - k0), dtype=torch.bool, device=DEV).triu(ahead + 1)
        for h in range(heads):
            at = h * s["kv_heads"] // heads
            z = s["queries"][q0:q1, h].double() @ s["keys"][k0:k1, at].double().t() * s["scale"]
            if s["causal"]:
                z[hidden] = -math.inf
            lse[q0:q1, h] = torch.logsumexp(z, -1)
            out[q0:q1, h] = torch.softmax(z, -1) @ s["values"][k0:k1, at].double()
    return out, lse


def exact_norm(s):
    h = s["x_in"].double() + (0 if s["res"] is None else s["res"].double())
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + EPS) * s["w"].double()
    codes, scales = torch.zeros_like(y), []
    grid = torch.arange(127, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    for part, place in zip(y.split(s["group"] or s["dim"], 1), codes.split(s["group"] or s["dim"], 1)):
        scale = part.abs().amax(-1, keepdim=True) / 448
        a = (part / scale.clamp(min=1e-300)).abs().contiguous()
        hi = torch.searchsorted(grid, a).clamp(1, 126)
        below, above = a - grid[hi - 1], grid[hi] - a
        at = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
        place.copy_(torch.copysign(grid[at], part))
        scales.append(scale)
    return codes, torch.cat(scales, 1), None if s["res"] is None else h


def exact_matvec(s):
    x, k = s["x_in"].double(), s["k"]
    if s["x_scales"] is not None:
        of = torch.arange(k, device=DEV) // 128
        x = x * s["x_scales"].double()[..., of]
    mag = torch.tensor(E2M1, device=DEV, dtype=torch.float64)
    y = torch.empty((s["tokens"], s["groups"], s["n"]), dtype=torch.float64, device=DEV)
    for g in range(s["groups"]):
        for n in range(0, s["n"], 4096):
            raw = s["codes"][g, n:n + 4096].long()
            nibble = torch.stack([raw % 16, raw // 16], -1).flatten(1)
            w = mag[nibble % 8] * (1 - 2 * (nibble // 8)) * s["scales"][g, n:n + 4096].double().repeat_interleave(16, 1)
            y[:, g, n:n + 4096] = x[:, g] @ w.t() * s["weight_scale"][g].double()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": exact_attend, "norm": exact_norm, "matvec": exact_matvec}[case["op"]](s)
