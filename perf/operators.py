"""Cases for the operators of the single-token path: linears with group-scaled 4-bit weights and
16-bit activations, the per-head norm and position rotation of queries and keys with the append to
the paged key-value cache, and the attention of one new token per sequence over that cache.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` is one pass,
through the library when ``own`` is set and in elementary torch operations (fp32 arithmetic, one
rounding at the end) otherwise, ``exact`` is the same result from the definition in fp64.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _linear(M, K, N, group, dtype, epi="none", **kw):
    return dict(op="linear", M=M, K=K, N=N, group=group, dtype=dtype, epi=epi, **kw)


def _rope(M, heads, kv_heads, D, rot, dtype, interleaved, page, far, pad=0, **kw):
    return dict(op="rope", M=M, heads=heads, kv_heads=kv_heads, D=D, rot=rot, dtype=dtype,
                interleaved=interleaved, page=page, far=far, pad=pad, **kw)


def _attn(B, heads, kv_heads, D, longest, page, dtype, window=0, sinks=0, **kw):
    return dict(op="attn", B=B, heads=heads, kv_heads=kv_heads, D=D, longest=longest, page=page,
                dtype=dtype, window=window, sinks=sinks, **kw)


def listed():
    return [
        # the small benchmark linear with its fp32 activations: a call that is all latency
        _linear(16, 256, 256, 64, "fp32", name="linear small fp32"),
        # one token through an attention-output projection, added to the residual
        _linear(1, 1024, 1024, 128, "fp16", "residual", name="linear one token"),
        # one token of a language backbone through its FFN up projection
        _linear(1, 2048, 16384, 64, "bf16", "gelu", name="linear one token wide"),
        # eight sequences decoded together through the long-K FFN down projection
        _linear(8, 16384, 2048, 128, "fp16", "residual", name="linear eight long-K"),
        # the 50 tokens of an action chunk, an output width that no tile divides, the smallest group
        _linear(50, 1024, 4099, 32, "bf16", name="linear chunk ragged N"),
        # one new token with a single shared key/value head
        _rope(1, 8, 1, 256, 256, "bf16", False, 16, 2000, name="rope one token"),
        # 32 episodes of 50 tokens, half of each head rotated in adjacent pairs, 37 padded rows
        _rope(1600, 16, 16, 64, 32, "fp16", True, 64, 1 << 15, pad=37, name="rope action chunks"),
        # a long prompt written to the cache at far positions
        _rope(8191, 32, 8, 128, 128, "bf16", False, 16, 1 << 20, name="rope long prompt"),
        # one token over a short cache with a single key/value head: latency
        _attn(1, 8, 1, 256, 1001, 16, "bf16", name="attn one short"),
        # a served batch with lengths from nothing to 8191
        _attn(32, 32, 8, 128, 8191, 64, "fp16", name="attn ragged batch"),
        # two long contexts
        _attn(2, 32, 8, 128, 131071, 256, "bf16", name="attn long"),
        # a batch of ordinary heads that sees 4 first tokens and the last 1000
        _attn(64, 16, 16, 64, 8000, 16, "fp16", window=1000, sinks=4, name="attn window"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "rope", "attn"])
    if op == "linear":
        group = rng.choice([32, 64, 128, 256])
        K = max(1, _log(rng, 256, 16384) // group) * group
        N = _log(rng, 100, min(16384, (1 << 25) // K))
        return _linear(_log(rng, 1, 64), K, N, group, rng.choice(["fp16", "bf16", "fp32"]),
                       rng.choice(["none", "gelu", "residual"]))
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 96, 128, 192, 256])
    dtype, page = rng.choice(["fp16", "bf16"]), rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        M = _log(rng, 1, (1 << 25) // ((heads + 2 * kv) * D))
        return _rope(M, heads, kv, D, rng.choice([D, D, D // 2]), dtype, rng.random() < 0.4, page,
                     _log(rng, M + 1, 1 << 20 if M < (1 << 19) else 1 << 21), rng.randrange(0, 1 + M // 8))
    B = _log(rng, 1, 96)
    longest = _log(rng, 1, max(2, (1 << 27) // (B * kv * D)))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return _attn(B, heads, kv, D, longest, page, dtype, window, rng.choice([0, 1, 4, 70]) if window else 0)


def _lengths(c):
    """The cache lengths of a batch, set by its case: the first is the longest, the others spread
    over a factor of 32 below it; a batch of eight or more also has a row of one token and an
    empty one."""
    rng = random.Random(c["B"] * 1000003 + c["longest"])
    out = [c["longest"]]
    while len(out) < c["B"]:
        out.append(_log(rng, max(1, c["longest"] // 32), c["longest"]))
    if c["B"] >= 8:
        out[3], out[5] = 1, 0
    return out


def _visible(c, n):
    """How many of n cached tokens the new token sees."""
    return n if c["window"] == 0 or n <= c["window"] else c["window"] + min(c["sinks"], n - c["window"])


def work(c):
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        xb = 4 if c["dtype"] == "fp32" else 2
        nbytes = N * K // 2 + 2 * N * (K // c["group"]) + M * K * xb + 2 * M * N
        return {"bytes": nbytes + (2 * M * N if c["epi"] == "residual" else 0), "flops": 2 * M * N * K}
    if c["op"] == "rope":
        n = c["M"] - c["pad"]
        rows = (c["heads"] + 2 * c["kv_heads"]) * c["D"]
        return {"bytes": 2 * n * rows * 2 + 2 * c["pad"] * c["heads"] * c["D"] * 2 + 16 * c["M"],
                "flops": c["M"] * (c["heads"] + c["kv_heads"]) * c["D"] * 7}
    seen = sum(_visible(c, n) for n in _lengths(c))
    return {"bytes": 2 * 2 * seen * c["kv_heads"] * c["D"] + 2 * 2 * c["B"] * c["heads"] * c["D"],
            "flops": 4 * seen * c["heads"] * c["D"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

# Byte i of an operand's dword holds the codes of these positions of its run of eight (low nibble,
# high nibble).
_LOW, _HIGH = [0, 4, 1, 5], [2, 6, 3, 7]


def _operand(codes):
    """The codes (int8 [N, K], -8..7) as the library's operand of a group-scaled linear: tiles of 16
    rows by 128 k, see w4a4_codes_to_w4g."""
    N, K = codes.shape
    n16, k128 = -(-N // 16), -(-K // 128)
    u = torch.full((n16 * 16, k128 * 128), 8, dtype=torch.uint8, device=codes.device)
    u[:N, :K] = (codes + 8).to(torch.uint8)
    u = u.view(n16, 16, k128, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)
    return (u[..., _LOW] | (u[..., _HIGH] << 4)).contiguous().view(-1)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "linear":
        M, K, N, group = c["M"], c["K"], c["N"], c["group"]
        ydt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
        W = (0.02 * normal(N, K)).view(N, K // group, group)
        s = (W.abs().amax(-1) / 7).half()
        codes = (W / s.float().unsqueeze(-1)).round().clamp(-8, 7).to(torch.int8).view(N, K)
        X = normal(M, K)
        X[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 15.0
        u = codes.to(torch.uint8) & 15
        return dict(c=c, X=X.to(dt), codes=u[:, 0::2] | (u[:, 1::2] << 4), operand=_operand(codes),
                    scale=s.t().contiguous(), residual=normal(M, N).to(ydt), ydt=ydt)
    if c["op"] == "rope":
        M, H, KV, D, page, rot = c["M"], c["heads"], c["kv_heads"], c["D"], c["page"], c["rot"]
        n = M - c["pad"]
        qkv = (normal(M, (H + 2 * KV) * D) * 2.0).to(dt)
        pages = -(-n // page) + 3
        slots = torch.full((M,), -1, dtype=torch.int64, device="cuda")
        perm = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        slots[:n] = perm[t // page] * page + t % page
        start = int(torch.randint(0, c["far"] - M, (1,), generator=g, device="cuda"))
        return dict(c=c, q=qkv[:, :H * D].view(M, H, D), k=qkv[:, H * D:(H + KV) * D].view(M, KV, D),
                    v=qkv[:, (H + KV) * D:].view(M, KV, D), qw=1 + 0.1 * normal(D), kw=1 + 0.1 * normal(D),
                    inv_freq=10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot),
                    positions=start + torch.arange(M, device="cuda"), slots=slots,
                    k_cache=torch.zeros(pages, KV, page, D, dtype=dt, device="cuda"),
                    v_cache=torch.zeros(pages, KV, page, D, dtype=dt, device="cuda"))
    B, H, KV, D, page = c["B"], c["heads"], c["kv_heads"], c["D"], c["page"]
    lens = _lengths(c)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 5
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    cache = [torch.randn(pages, KV, page, D, dtype=dt, generator=g, device="cuda") for _ in range(2)]
    return dict(c=c, q=(1.5 * normal(B, H, D)).to(dt), k_cache=cache[0], v_cache=cache[1], table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _plain_linear(s):
    c, codes = s["c"], s["codes"]
    N, K, group = c["N"], c["K"], c["group"]
    u = torch.stack((codes & 15, codes >> 4), -1).view(N, K // group, group)
    v = (u ^ 8).float() - 8
    W = (v * s["scale"].t().float().unsqueeze(-1)).view(N, K)
    y = s["X"].float() @ W.t()
    if c["epi"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["epi"] == "residual":
        y = y + s["residual"].float()
    return y.to(s["ydt"])


def _plain_rotate(x, w, cos, sin, rot, interleaved):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _plain_rope(s):
    c, dt = s["c"], s["q"].dtype
    angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    q = _plain_rotate(s["q"], s["qw"], cos, sin, c["rot"], c["interleaved"]).to(dt)
    k = _plain_rotate(s["k"], s["kw"], cos, sin, c["rot"], c["interleaved"]).to(dt)
    n = c["M"] - c["pad"]
    page, off = s["slots"][:n] // c["page"], s["slots"][:n] % c["page"]
    s["k_cache"][page, :, off] = k[:n]
    s["v_cache"][page, :, off] = s["v"][:n]
    return q, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    c = s["c"]
    B, H, KV, D, page = c["B"], c["heads"], c["kv_heads"], c["D"], c["page"]
    n = s["lens"].long().unsqueeze(1)
    if c["window"] and c["window"] + c["sinks"] < c["longest"]:
        first = torch.arange(c["sinks"], device="cuda").expand(B, -1)
        last = n - c["window"] + torch.arange(c["window"], device="cuda")
        keys = torch.cat((first, last), 1)
        seen = torch.cat((first < n, last >= c["sinks"]), 1) & (keys < n)
        keys = keys.clamp(min=0)
    else:
        keys = torch.arange(c["longest"], device="cuda").expand(B, -1)
        seen = keys < n
    ids = s["table"].long().gather(1, (keys // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    heads = torch.arange(KV, device="cuda").view(1, KV, 1)
    at = (ids.unsqueeze(1), heads, (keys % page).unsqueeze(1))
    k, v = s["k_cache"][at].float(), s["v_cache"][at].float()
    score = (s["q"].float().view(B, KV, H // KV, D) * s["scale"]) @ k.transpose(-1, -2)
    score = score.masked_fill(~seen.view(B, 1, 1, -1), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.masked_fill(total == 0, 1.0)
    return out.view(B, H, D).to(s["q"].dtype)


def run(s):
    c = s["c"]
    if not own:
        return {"linear": _plain_linear, "rope": _plain_rope, "attn": _plain_attn}[c["op"]](s)
    from w4a4_post_quantized_zigzag_amd import binding as bd
    if c["op"] == "linear":
        epi = {"none": bd.EPI_NONE, "gelu": bd.EPI_GELU, "residual": bd.EPI_RESIDUAL}[c["epi"]]
        return bd.gemv_w4g(s["X"], s["operand"], s["scale"], epilogue=epi,
                           residual=s["residual"] if c["epi"] == "residual" else None)
    if c["op"] == "rope":
        q = bd.qk_norm_rope_append(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["inv_freq"], s["positions"],
                                   s["k_cache"], s["v_cache"], s["slots"], eps=_EPS,
                                   interleaved=c["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    return bd.paged_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=s["scale"],
                                window=c["window"], sinks=c["sinks"], max_len=c["longest"])


# ---------------------------------------------------------------------------------------------
# the definition, in fp64
# ---------------------------------------------------------------------------------------------

def _exact_linear(s):
    c, codes = s["c"], s["codes"]
    M, N, K, group = c["M"], c["N"], c["K"], c["group"]
    value = torch.tensor([i if i < 8 else i - 16 for i in range(16)], dtype=torch.float64, device="cuda")
    x = s["X"].double()
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for k0 in range(0, K, 1024):  # a slab of columns at a time, group by group inside it
        part = codes[:, k0 // 2:(k0 + 1024) // 2].long()
        w = torch.empty(N, 2 * part.shape[1], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = value[part % 16], value[part // 16]
        for j in range(0, w.shape[1], group):
            y += (x[:, k0 + j:k0 + j + group] @ w[:, j:j + group].t().contiguous()) * s["scale"][(k0 + j) // group].double()
    if c["epi"] == "gelu":
        y = y * torch.special.ndtr(y)
    return y + s["residual"].double() if c["epi"] == "residual" else y


def _exact_rotate(x, w, positions, inv_freq, rot, interleaved):
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt() * w.double()
    turn = torch.polar(torch.ones_like(inv_freq), positions.double().outer(inv_freq)).unsqueeze(1)
    if interleaved:
        z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["c"]
    q = _exact_rotate(s["q"], s["qw"], s["positions"], s["inv_freq"], c["rot"], c["interleaved"])
    k = _exact_rotate(s["k"], s["kw"], s["positions"], s["inv_freq"], c["rot"], c["interleaved"])
    rows = [(r, t) for r, t in enumerate(s["slots"].tolist()) if t >= 0]
    r, t = (torch.tensor(v, device="cuda") for v in zip(*rows))
    P, KV, page, D = s["k_cache"].shape
    caches = []
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
        flat = cache.double().transpose(1, 2).reshape(P * page, KV, D)
        flat[t] = new[r]
        caches.append(flat.view(P, page, KV, D).transpose(1, 2).contiguous())
    return q, caches[0], caches[1]


def _exact_attn(s):
    c = s["c"]
    H, KV, D, page = c["heads"], c["kv_heads"], c["D"], c["page"]
    out = torch.zeros(c["B"], H, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        if c["window"]:
            j = j[(j < c["sinks"]) | (j >= n - c["window"])]
        if not len(j):
            continue
        ids = s["table"][b].long()[j // page]
        for h in range(KV):
            k, v = s["k_cache"][ids, h, j % page].double(), s["v_cache"][ids, h, j % page].double()
            q = s["q"][b, h * (H // KV):(h + 1) * (H // KV)].double()
            out[b, h * (H // KV):(h + 1) * (H // KV)] = torch.softmax(q @ k.t().contiguous() * s["scale"], -1) @ v
    return out


def exact(c, seed):
    s = prepare(c, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "attn": _exact_attn}[c["op"]](s)
