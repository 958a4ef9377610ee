"""Cases for the operators around a quantized key-value cache and around shared work of a served batch:
the per-head norm and rotation with an append that quantizes, and the rows read back; the attention of
one new token per sequence over that cache; the same attention for a batch whose sequences begin with
one shared prefix; and low-rank adapters of many requests beside a shared projection.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` is one pass,
through the library when ``own`` is set and in elementary torch operations (fp32 arithmetic, one
rounding at the end) otherwise, ``exact`` is the same result from the definition in fp64.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-6
# E2M1 magnitudes by code
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# exponents of a block's scale: every value is then exact and finite in the element type
_FP4_RANGE = {torch.float16: (-23, 13), torch.bfloat16: (-100, 125)}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _cache(M, heads, kv_heads, D, rot, dtype, kind, interleaved, page, far, pad=0, **kw):
    return dict(op="cache", M=M, heads=heads, kv_heads=kv_heads, D=D, rot=rot, dtype=dtype, kind=kind,
                interleaved=interleaved, page=page, far=far, pad=pad, **kw)


def _attn(B, heads, kv_heads, D, longest, page, dtype, kind, window=0, sinks=0, **kw):
    return dict(op="attn", B=B, heads=heads, kv_heads=kv_heads, D=D, longest=longest, page=page,
                dtype=dtype, kind=kind, window=window, sinks=sinks, prefix=0, **kw)


def _shared(B, heads, kv_heads, D, prefix, longest, page, dtype, kind, **kw):
    return dict(op="shared", B=B, heads=heads, kv_heads=kv_heads, D=D, prefix=prefix, longest=longest,
                page=page, dtype=dtype, kind=kind, window=0, sinks=0, **kw)


def _adapter(M, K, N, R, n, dtype, epi="none", run=1, **kw):
    return dict(op="adapter", M=M, K=K, N=N, R=R, n=n, dtype=dtype, epi=epi, run=run, **kw)


def listed():
    return [
        # one new token with a single shared key/value head, written in 8 bits and read back
        _cache(1, 8, 1, 256, 256, "bf16", "int8", False, 16, 2000, name="cache one token int8"),
        # 32 episodes of 50 tokens, half of each head rotated in adjacent pairs, 37 padded rows
        _cache(1600, 16, 16, 64, 32, "fp16", "int8", True, 64, 1 << 15, pad=37, name="cache action chunks int8"),
        # a long prompt written in 4 bits at far positions, and read back for the next chunk of it
        _cache(8191, 32, 8, 128, 128, "bf16", "fp4", False, 16, 1 << 20, name="cache long prompt fp4"),
        # one token over a short cache with a single key/value head: latency
        _attn(1, 8, 1, 256, 1001, 16, "bf16", "int8", name="attn one short int8"),
        # a served batch with lengths from nothing to 8191
        _attn(32, 32, 8, 128, 8191, 64, "fp16", "int8", name="attn ragged batch int8"),
        # two long contexts
        _attn(2, 32, 8, 128, 131071, 256, "bf16", "fp4", name="attn long fp4"),
        # eight action chunks behind one instruction of 600 tokens: latency
        _shared(8, 8, 1, 256, 600, 50, 16, "fp16", "none", name="shared instruction"),
        # a served batch behind one long system prompt
        _shared(64, 32, 8, 128, 16384, 700, 64, "bf16", "none", name="shared long prompt"),
        # the same kind of batch over a quantized cache, a prefix that ends inside a page
        _shared(48, 16, 2, 128, 30011, 1500, 32, "fp16", "int8", name="shared prompt int8"),
        # one request with its adapter at an attention-output projection
        _adapter(1, 1024, 1024, 16, 4, "fp16", "residual", name="adapter one token"),
        # 32 decoded requests, mostly with adapters of their own, at an FFN up projection
        _adapter(32, 2048, 16384, 16, 24, "bf16", "gelu", name="adapter served batch"),
        # 32 episodes of 50 tokens, each with one adapter, an output width that no tile divides
        _adapter(1600, 1024, 4099, 64, 32, "fp16", "none", run=50, name="adapter action chunks"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "attn", "shared", "adapter"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "adapter":
        M, run = rng.choice([(_log(rng, 1, 96), 1), (_log(rng, 97, 2048), rng.choice([1, 7, 50, 400]))])
        K, N = 8 * _log(rng, 16, 1024), _log(rng, 100, 16384 if M < 97 else 4099)
        R = rng.choice([8, 16, 24, 32, 64, 128])
        n = _log(rng, 1, max(2, min(48, (1 << 25) // ((K + N) * R))))
        return _adapter(M, K, N, R, n, dtype, rng.choice(["none", "gelu", "residual"]), run)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    D, page = rng.choice([64, 96, 128, 192, 256]), rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["int8", "fp4"])
    if op == "cache":
        M = _log(rng, 1, (1 << 25) // ((heads + 2 * kv) * D))
        return _cache(M, heads, kv, D, rng.choice([D, D, D // 2]), dtype, kind, rng.random() < 0.4, page,
                      _log(rng, M + 1, 1 << 21), rng.randrange(0, 1 + M // 8))
    if op == "attn":
        B = _log(rng, 1, 96)
        longest = _log(rng, 1, max(2, (1 << 27) // (B * kv * D)))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return _attn(B, heads, kv, D, longest, page, dtype, kind, window, rng.choice([0, 1, 4, 70]) if window else 0)
    B = _log(rng, 1, 96)
    prefix = _log(rng, 16, max(17, min(65536, (3 << 24) // (kv * D), (1 << 32) // (B * heads * D))))
    longest = _log(rng, 1, max(2, min(prefix, (1 << 23) // (B * kv * D))))
    return _shared(B, heads, kv, D, prefix, longest, page, dtype, rng.choice(["none", "none", kind]))


def _lengths(c):
    """The lengths of a batch's own tokens, set by its case: the first is the longest, the others spread
    over a factor of 32 below it; a batch of eight or more also has a row of one token and an
    empty one."""
    rng = random.Random(c["B"] * 1000003 + c["longest"])
    out = [c["longest"]]
    while len(out) < c["B"]:
        out.append(_log(rng, max(1, c["longest"] // 32), c["longest"]))
    if c["B"] >= 8:
        out[3], out[5] = 1, 0
    return out


def _ids(c):
    """Each row's adapter, set by its case: runs of rows with one adapter, about one in ten with none."""
    rng = random.Random(c["M"] * 1000003 + c["n"])
    out = []
    while len(out) < c["M"]:
        out += [-1 if out and rng.random() < 0.1 else rng.randrange(c["n"])] * c["run"]
    return out[:c["M"]]


def _visible(c, n):
    """How many of n cached tokens the new token sees."""
    return n if c["window"] == 0 or n <= c["window"] else c["window"] + min(c["sinks"], n - c["window"])


def _row_bytes(kind, D):
    """Bytes of one token's key (or value) of one head in the cache."""
    return {"none": 2 * D, "int8": D + 4, "fp4": D // 2 + D // 32}[kind]


def work(c):
    if c["op"] == "adapter":
        M, K, N, R = c["M"], c["K"], c["N"], c["R"]
        ids = _ids(c)
        rows = sum(i >= 0 for i in ids)
        nbytes = 2 * (len(set(ids) - {-1}) * R * (K + N) + rows * K + 2 * M * N)
        return {"bytes": nbytes + (2 * M * N if c["epi"] == "residual" else 0), "flops": 2 * rows * R * (K + N)}
    H, KV, D = c["heads"], c["kv_heads"], c["D"]
    row = _row_bytes(c["kind"], D)
    if c["op"] == "cache":
        n = c["M"] - c["pad"]
        # rows in, queries out, codes and scales written and read, rows out
        return {"bytes": 2 * c["M"] * (H + 2 * KV) * D + 2 * c["M"] * H * D + 4 * n * KV * row + 4 * c["M"] * KV * D,
                "flops": c["M"] * (H + KV) * D * 7}
    seen = [_visible(c, n) for n in _lengths(c)]
    return {"bytes": 2 * (c["prefix"] + sum(seen)) * KV * row + 2 * 2 * c["B"] * H * D,
            "flops": 4 * (c["prefix"] * c["B"] + sum(seen)) * H * D}


# ---------------------------------------------------------------------------------------------
# the two formats of a quantized row: codes and scales, and the values they stand for
# ---------------------------------------------------------------------------------------------

def _quantize(x, kind):
    """Rows x [..., D] (16-bit). int8: codes int8 [..., D] and an fp32 scale [...]; fp4: two E2M1 codes per
    byte, the even channel low, [..., D / 2] and the exponent byte of each 32 channels' scale [..., D / 32]."""
    f = x.float()
    if kind == "int8":
        m = f.abs().amax(-1).clamp(min=2.0 ** -100)
        return torch.round(f * (127.0 / m).unsqueeze(-1)).to(torch.int8), m / 127.0
    f = f.unflatten(-1, (-1, 32))
    fraction, e = torch.frexp(f.abs().amax(-1))
    e = torch.where(fraction > 0.75, e - 2, e - 3).clamp(*_FP4_RANGE[x.dtype])
    y = torch.ldexp(f, -e.unsqueeze(-1)).abs()
    y = torch.where(y < 2, torch.round(2 * y) / 2, torch.where(y < 4, torch.round(y), 2 * torch.round(y / 2))).clamp(max=6.0)
    code = torch.where(y < 2, 2 * y, torch.where(y < 4, y + 2, y / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(f).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scale, kind):
    """fp32 values of codes and scales."""
    if kind == "none":
        return codes.float()
    if kind == "int8":
        return codes.float() * scale.unsqueeze(-1)
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=codes.device)[u.long()]
    return torch.ldexp(v.unflatten(-1, (-1, 32)), scale.int().unsqueeze(-1) - 127).flatten(-2)


def _pages(kind, pages, KV, page, D, dt):
    """An empty cache: (k, v) of 16-bit elements, or (k, v, k_scale, v_scale)."""
    z = lambda shape, t: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    if kind == "none":
        return tuple(z((pages, KV, page, D), dt) for _ in range(2))
    if kind == "int8":
        return tuple(z((pages, KV, page, D), torch.int8) for _ in range(2)) + tuple(
            z((pages, KV, page), torch.float32) for _ in range(2))
    return tuple(z((pages, KV, page, D // 2), torch.uint8) for _ in range(2)) + tuple(
        z((pages, KV, D // 32, page), torch.uint8) for _ in range(2))


def _gather(cache, which, kind, at):
    """Values of keys (0) or values (1) at (page, head, offset) index tensors."""
    if kind == "none":
        return cache[which][at].float()
    scale = cache[2 + which]
    if kind == "fp4":
        scale = scale.transpose(2, 3)
    return _values(cache[which][at], scale[at], kind)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "adapter":
        M, K, N, R, n = c["M"], c["K"], c["N"], c["R"], c["n"]
        X = normal(M, K)
        X[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 15.0
        return dict(c=c, X=X.to(dt), A=(normal(n, R, K) * K ** -0.5).to(dt), Bm=(0.1 * normal(n, N, R)).to(dt),
                    ids=torch.tensor(_ids(c), dtype=torch.int32, device="cuda"),
                    scale=0.5 + torch.rand(n, generator=g, device="cuda"), Y=normal(M, N).to(dt),
                    residual=normal(M, N).to(dt))
    H, KV, D, page, kind = c["heads"], c["kv_heads"], c["D"], c["page"], c["kind"]
    if c["op"] == "cache":
        M, rot = c["M"], c["rot"]
        n = M - c["pad"]
        qkv = normal(M, (H + 2 * KV) * D) * 2.0
        qkv[:, torch.randperm((H + 2 * KV) * D, generator=g, device="cuda")[:(H + 2 * KV) * D // 50]] *= 6.0
        qkv = qkv.to(dt)
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
                    cache=_pages(kind, pages, KV, page, D, dt))
    B, lens = c["B"], _lengths(c)
    used = [-(-n // page) for n in lens]
    front = -(-c["prefix"] // page)
    pages = front + sum(used) + 5
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = front
    for b, n in enumerate(used):
        table[b, :n] = ids[at:at + n]
        at += n
    rows = [torch.randn(pages, KV, page, D, dtype=dt, generator=g, device="cuda") for _ in range(2)]
    if kind != "none":
        (k, ks), (v, vs) = (_quantize(x, kind) for x in rows)
        if kind == "fp4":
            ks, vs = (s.transpose(2, 3).contiguous() for s in (ks, vs))
        rows = (k, v, ks, vs)
    return dict(c=c, q=(1.5 * normal(B, H, D)).to(dt), cache=tuple(rows), table=table, prefix_table=ids[:front],
                prefix_len=torch.tensor([c["prefix"]], dtype=torch.int32, device="cuda"),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=D ** -0.5)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _plain_rotate(x, w, cos, sin, rot, interleaved):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _plain_cache(s):
    c, dt, kind = s["c"], s["q"].dtype, s["c"]["kind"]
    angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"]
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    q = _plain_rotate(s["q"], s["qw"], cos, sin, c["rot"], c["interleaved"]).to(dt)
    k = _plain_rotate(s["k"], s["kw"], cos, sin, c["rot"], c["interleaved"]).to(dt)
    n = c["M"] - c["pad"]
    page, off = s["slots"][:n] // c["page"], s["slots"][:n] % c["page"]
    back = []
    heads = torch.arange(c["kv_heads"], device="cuda")
    at = (page.unsqueeze(1), heads, off.unsqueeze(1))
    for which, x in ((0, k), (1, s["v"])):
        codes, scale = _quantize(x[:n], kind)
        s["cache"][which][at] = codes
        held = s["cache"][2 + which]
        (held if kind == "int8" else held.transpose(2, 3))[at] = scale
        rows = torch.zeros_like(x)
        rows[:n] = _gather(s["cache"], which, kind, at).to(dt)
        back.append(rows)
    return q, back[0], back[1]


def _plain_scores(c, s):
    """Visible tokens of each sequence: their keys and values, and the scores [B, KV, G, tokens]."""
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
    k, v = (_gather(s["cache"], i, c["kind"], at) for i in range(2))
    score = (s["q"].float().view(B, KV, H // KV, D) * s["scale"]) @ k.transpose(-1, -2)
    return score.masked_fill(~seen.view(B, 1, 1, -1), -math.inf), v


def _plain_attn(s):
    c = s["c"]
    score, v = _plain_scores(c, s)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.masked_fill(total == 0, 1.0)
    return out.view(c["B"], c["heads"], c["D"]).to(s["q"].dtype)


def _plain_shared(s):
    c = s["c"]
    B, H, KV, D, page, P = c["B"], c["heads"], c["kv_heads"], c["D"], c["page"], c["prefix"]
    score, v = _plain_scores(c, s)
    keys = torch.arange(P, device="cuda")
    at = (s["prefix_table"].long()[keys // page], torch.arange(KV, device="cuda").view(KV, 1), keys % page)
    pk, pv = (_gather(s["cache"], i, c["kind"], at) for i in range(2))
    q = s["q"].float().view(B, KV, H // KV, D).transpose(0, 1).reshape(KV, -1, D) * s["scale"]
    ps = q @ pk.transpose(-1, -2)  # all sequences' queries at once
    score, v = score.transpose(0, 1), v.transpose(0, 1)
    own_top = score.amax(-1, keepdim=True)
    top = torch.maximum(ps.view(KV, B, H // KV, P).amax(-1, keepdim=True), own_top)
    pp = torch.exp(ps - top.view(KV, -1, 1))
    p = torch.exp(score - top)
    out = (pp @ pv).view(KV, B, H // KV, D) + p @ v
    out = out / (pp.sum(-1).view(KV, B, H // KV, 1) + p.sum(-1, keepdim=True))
    return out.transpose(0, 1).reshape(B, H, D).to(s["q"].dtype)


def _plain_adapter(s):
    c = s["c"]
    M, N, R, n = c["M"], c["N"], c["R"], c["n"]
    mine = (s["ids"].unsqueeze(1) == torch.arange(n, device="cuda")).float() * s["scale"]
    t = (s["X"].float() @ s["A"].float().view(n * R, -1).t()).view(M, n, R) * mine.unsqueeze(-1)
    y = s["Y"].float() + t.view(M, n * R) @ s["Bm"].float().transpose(1, 2).reshape(n * R, N)
    if c["epi"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["epi"] == "residual":
        y = y + s["residual"].float()
    return y.to(s["Y"].dtype)


def run(s):
    c = s["c"]
    if not own:
        return {"cache": _plain_cache, "attn": _plain_attn, "shared": _plain_shared,
                "adapter": _plain_adapter}[c["op"]](s)
    from w4a4_post_quantized_zigzag_amd import binding as bd
    if c["op"] == "adapter":
        epi = {"none": bd.EPI_NONE, "gelu": bd.EPI_GELU, "residual": bd.EPI_RESIDUAL}[c["epi"]]
        return bd.adapter_add(s["Y"], s["X"], s["A"], s["Bm"], s["ids"], s["scale"], epilogue=epi,
                              residual=s["residual"] if c["epi"] == "residual" else None)
    if c["op"] == "cache":
        q = bd.qk_norm_rope_append_quant(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["inv_freq"], s["positions"],
                                         s["cache"], s["slots"], eps=_EPS, interleaved=c["interleaved"])
        k, v = bd.kv_read_quant(s["cache"], s["slots"], s["q"].dtype)
        return q, k, v
    if c["op"] == "attn":
        return bd.paged_attn_decode_quant(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"],
                                          window=c["window"], sinks=c["sinks"], max_len=c["longest"])
    return bd.paged_attn_shared(s["q"], s["cache"], s["prefix_table"], s["prefix_len"], s["table"], s["lens"],
                                scale=s["scale"], max_prefix=c["prefix"], max_len=c["longest"])


# ---------------------------------------------------------------------------------------------
# the definition, in fp64
# ---------------------------------------------------------------------------------------------

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


def _exact_quantized(y, kind, dt):
    """The values that rows y [..., D] are held as."""
    if kind == "int8":
        s = y.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 127
        return (y / s).round() * s
    g = y.view(*y.shape[:-1], -1, 32)
    s = torch.exp2((g.abs().amax(-1, keepdim=True) / 6).log2().ceil().clamp(*_FP4_RANGE[dt]))
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=y.device)
    a = (g / s).abs()
    hi = torch.searchsorted(grid, a.clamp(max=6.0)).clamp(max=7)  # first code that is not below
    lo = (hi - 1).clamp(min=0)
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    return (torch.where(up, grid[hi], grid[lo]) * g.sign() * s).view(y.shape)


def _exact_cache(s):
    c, kind, dt = s["c"], s["c"]["kind"], s["q"].dtype
    q = _exact_rotate(s["q"], s["qw"], s["positions"], s["inv_freq"], c["rot"], c["interleaved"])
    k = _exact_rotate(s["k"], s["kw"], s["positions"], s["inv_freq"], c["rot"], c["interleaved"])
    kept = (s["slots"] >= 0).view(-1, 1, 1)
    return q, _exact_quantized(k, kind, dt) * kept, _exact_quantized(s["v"].double(), kind, dt) * kept


def _exact_rows(s, which, kind, ids, h, off):
    x = s["cache"][which][ids, h, off]
    if kind == "none":
        return x.double()
    if kind == "int8":
        return x.double() * s["cache"][2 + which][ids, h, off].double().unsqueeze(-1)
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    full = torch.empty(x.shape[0], 2 * x.shape[1], dtype=torch.float64, device=x.device)
    for half, u in ((0, x % 16), (1, x // 16)):
        full[:, half::2] = grid[(u % 8).long()] * (1 - 2.0 * (u // 8))
    e = s["cache"][2 + which][ids, h, :, off].double() - 127
    return full * torch.exp2(e).repeat_interleave(32, -1)


def _exact_attn(s):
    c, kind = s["c"], s["c"]["kind"]
    H, KV, D, page = c["heads"], c["kv_heads"], c["D"], c["page"]
    G = H // KV
    out = torch.zeros(c["B"], H, D, dtype=torch.float64, device="cuda")
    t = torch.arange(c["prefix"], device="cuda")
    for h in range(KV):
        if c["prefix"]:
            ids = s["prefix_table"].long()[t // page]
            pk, pv = (_exact_rows(s, i, kind, ids, h, t % page) for i in range(2))
            pk = pk.t().contiguous()
        for b, n in enumerate(s["lens"].tolist()):
            j = torch.arange(n, device="cuda")
            if c["window"]:
                j = j[(j < c["sinks"]) | (j >= n - c["window"])]
            if not len(j) and not c["prefix"]:
                continue
            q = s["q"][b, h * G:(h + 1) * G].double()
            ids = s["table"][b].long()[j // page]
            k, v = (_exact_rows(s, i, kind, ids, h, j % page) for i in range(2))
            score = q @ k.t().contiguous()
            if c["prefix"]:
                p = torch.softmax(torch.cat((q @ pk, score), -1) * s["scale"], -1)
                out[b, h * G:(h + 1) * G] = p[:, :c["prefix"]].contiguous() @ pv + p[:, c["prefix"]:].contiguous() @ v
            else:
                out[b, h * G:(h + 1) * G] = torch.softmax(score * s["scale"], -1) @ v
    return out


def _exact_adapter(s):
    c = s["c"]
    y = s["Y"].double()
    for i in sorted(set(s["ids"].tolist()) - {-1}):
        rows = (s["ids"] == i).nonzero().flatten()
        inner = s["X"][rows].double() @ s["A"][i].double().t().contiguous()
        y[rows] += s["scale"][i].double() * (inner @ s["Bm"][i].double().t().contiguous())
    if c["epi"] == "gelu":
        return y * torch.special.ndtr(y)
    return y + s["residual"].double() if c["epi"] == "residual" else y


def exact(c, seed):
    s = prepare(c, seed)
    return {"cache": _exact_cache, "attn": _exact_attn, "shared": _exact_attn, "adapter": _exact_adapter}[c["op"]](s)
