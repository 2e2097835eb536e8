"""Workloads of the operators around a paged KV cache: the norm and rotation of new
queries and keys, the append of new tokens, and the attention of a batch over a shared
prefix.  Each has its plain form (elementary torch operations in 32 bits) and, where
`own` is true, the library's call.

Sizes follow the seeded workloads of this repository (8 KV and 64 query heads of 128,
latent rows of 576, histories of 32K and 128K) or are generic ragged ones.
"""

import math

import torch

own = False

ROPE_BASE = 500000.0
BLOCK = 16


def listed():
    return [
        # one new token for each of 8 requests between the projection and the cache: all latency
        dict(name="rope_decode_8", op="rope", tokens=8, H=8, Hq=64, d=128, dtype="bf16", rot=128, style="half",
             norm=True, span=32768),
        # a prefill batch through one layer: all bandwidth
        dict(name="rope_prefill_8192", op="rope", tokens=8192, H=8, Hq=64, d=128, dtype="bf16", rot=128,
             style="half", norm=True, span=131072),
        # an odd count of tokens in fp32, a partial rotation in adjacent pairs, groups of five
        dict(name="rope_odd_f32", op="rope", tokens=1237, H=8, Hq=40, d=128, dtype="f32", rot=64, style="pair",
             norm=True, span=1048576),
        # one new token for each of 64 requests into the cache
        dict(name="append_decode_64", op="append", batch=64, longest=500, decode=True, tokens=64, H=8, Hq=64, d=128,
             dtype="bf16", rot=128, style="half", norm=True),
        # chunks of five requests in one call, padded at the end as a serving loop does
        dict(name="append_chunks_4099", op="append", batch=5, longest=2000, decode=False, tokens=4099, H=8, Hq=64,
             d=128, dtype="bf16", rot=128, style="half", norm=True),
        # latent rows: the norm covers the 512 latent entries, the rotation the last 64
        dict(name="append_latent_2048", op="append", batch=4, longest=700, decode=False, tokens=2048, H=1, Hq=128,
             d=576, dtype="bf16", rot=64, style="pair", norm=True),
        # four requests, a short prefix and shorter tails: all latency
        dict(name="prefix_b4_777", op="prefix", batch=4, H=8, Hq=64, prefix=777, tail=90, empty=0),
        # the serving batch of 8 on a 32K prompt
        dict(name="prefix_b8_32k", op="prefix", batch=8, H=8, Hq=64, prefix=32768, tail=512, empty=0),
        # odd everything: 29 requests, two of them finished, groups of 7, long tails
        dict(name="prefix_b29_10007", op="prefix", batch=29, H=4, Hq=28, prefix=10007, tail=2500, empty=2),
        # a batch of 64 on a 128K prefix: more arithmetic than bytes
        dict(name="prefix_b64_128k", op="prefix", batch=64, H=8, Hq=64, prefix=131072, tail=1000, empty=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix"])
    H = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 6000), H=H, Hq=H * G, d=128, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rot=rng.choice([32, 64, 128]), style=rng.choice(["half", "pair"]),
                    norm=rng.random() < 0.75, span=_log(rng, 1000, 1048576))
    if op == "append":
        latent = rng.random() < 0.25
        decode = rng.random() < 0.4
        batch = _log(rng, 1, 64) if decode else rng.randint(1, 8)
        longest = _log(rng, 20, 2000) if not decode else _log(rng, 20, 600)
        return dict(op=op, batch=batch, longest=longest, decode=decode,
                    tokens=batch if decode else rng.randint(1, batch * longest),
                    H=1 if latent else H, Hq=128 if latent else H * G, d=576 if latent else 128,
                    dtype="bf16" if latent else rng.choice(["bf16", "bf16", "f32"]),
                    rot=64 if latent else rng.choice([32, 64, 128]), style=rng.choice(["half", "pair"]),
                    norm=rng.random() < 0.75)
    batch = _log(rng, 1, 64)
    return dict(op=op, batch=batch, H=H, Hq=H * G, prefix=_log(rng, 1, 100000), tail=_log(rng, 1, 1000),
                empty=rng.randint(0, batch // 8))


# ---------------------------------------------------------------------------- inputs


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int64)


def _rotation(case, g, dtype):
    """Rotation frequencies and the norm's weights; None for the weights of a model without the norm."""
    r = case["rot"]
    inv = (ROPE_BASE ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(torch.float32).cuda()
    n = case["d"] if case["d"] != 576 else 512
    gq = gk = None
    if case["norm"]:
        gk = (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dtype)
        if case["d"] != 576:  # latent queries are absorbed: rotated, not normed
            gq = (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dtype)
    return inv, gq, gk


def _qkv(case, g, dtype, v):
    """The projection's fused output, one row a token; q, k and v are column ranges of it."""
    n, H, Hq, d = case["tokens"], case["H"], case["Hq"], case["d"]
    row = _normal((n, (Hq + (2 if v else 1) * H) * d), g, dtype)
    q = row[:, :Hq * d].view(n, Hq, d)
    k = row[:, Hq * d:(Hq + H) * d].view(n, H, d)
    return q, k, row[:, (Hq + H) * d:].view(n, H, d) if v else None


def _pool(blocks, H, bs, d, g, dtype):
    return _normal((blocks, H, bs, d), g, dtype)


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case=case)
    if case["op"] == "prefix":
        return _prepare_prefix(case, g, s)
    dtype = _dtype(case)
    s["inv"], s["gq"], s["gk"] = _rotation(case, g, dtype)
    n, H, Hq, d = case["tokens"], case["H"], case["Hq"], case["d"]
    latent = d == 576
    s["q"], s["k"], s["v"] = _qkv(case, g, dtype, v=case["op"] == "append" and not latent)
    s["q_out"] = torch.zeros((n, Hq, d), dtype=dtype, device="cuda")  # padding tokens are never written
    if case["op"] == "rope":
        s["k_out"] = torch.empty((n, H, d), dtype=dtype, device="cuda")
        s["positions"] = _ints(0, case["span"], (n,), g).to(torch.int32)
        s["requests"] = None
        B, cap, bs = 1, case["span"], BLOCK
        lens = torch.full((1,), case["span"], dtype=torch.int32, device="cuda")
    else:
        B, cap, bs = case["batch"], case["longest"], 1 if latent else BLOCK
        per = (cap + bs - 1) // bs
        s["table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        s["pool_k"] = _pool(B * per, H, bs, d, g, dtype)
        s["pool_v"] = None if latent else _pool(B * per, H, bs, d, g, dtype)
        if case["decode"]:
            lens = _ints(0, cap + 1, (B,), g).to(torch.int32)  # a length of 0: an unused row of the batch
            s["positions"] = s["requests"] = None  # token i ends request i's history
        else:
            # every request's chunk ends its history; the tokens past the last chunk are padding
            share = n // B
            ids = torch.arange(n, device="cuda") // max(share, 1)
            lens = _ints(max(share, 1), cap + 1, (B,), g).to(torch.int32) if share else torch.full(
                (B,), cap, dtype=torch.int32, device="cuda")
            real = ids < B if share else torch.arange(n, device="cuda") < 0
            ids = ids.clamp(max=B - 1)
            at = lens.long()[ids] - share + torch.arange(n, device="cuda") % max(share, 1)
            s["positions"] = torch.where(real, at, -1).to(torch.int32)
            s["requests"] = torch.where(real, ids, -1).to(torch.int32)
    s["seq_lens"], s["bs"] = lens, bs
    if own:
        import top_sparse_kv_gb300 as skv

        p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=512 if latent else d, max_len=cap, topk=0,
                        n_sink=0, n_local=0, block_size=bs, seq_lens=lens,
                        dtype=skv.SKV_DTYPE_F32 if dtype == torch.float32 else skv.SKV_DTYPE_BF16)
        rot = skv.Rotary(inv_freq=s["inv"], rot_dim=case["rot"], rot_start=512 if latent else 0,
                         style=skv.SKV_ROPE_HALF if case["style"] == "half" else skv.SKV_ROPE_PAIR,
                         norm_dim=512 if latent else d, eps=1e-6, q_gamma=s["gq"], k_gamma=s["gk"])
        pool = skv.Pool(s["pool_k"], s["pool_v"], s["table"]) if case["op"] == "append" else None
        s["step"] = skv.TokenStep(p, rot, pool)
    return s


def _prepare_prefix(case, g, s):
    B, H, Hq, P, tail = case["batch"], case["H"], case["Hq"], case["prefix"], case["tail"]
    d, bs = 128, BLOCK
    lens = P + _ints(0, tail + 1, (B,), g)
    order = torch.randperm(B, generator=g, device="cuda")
    lens = torch.where(torch.isin(torch.arange(B, device="cuda"), order[:case["empty"]]), 0, lens)
    cap = P + tail
    per = (cap + bs - 1) // bs
    shared, tails = (P + bs - 1) // bs, per - P // bs  # the prefix's blocks; each request's own from P / bs on
    perm = torch.randperm(shared + B * tails, generator=g, device="cuda").to(torch.int32)
    s["prefix_table"] = perm[:shared].contiguous()
    table = torch.empty((B, per), dtype=torch.int32, device="cuda")
    table[:, :P // bs] = s["prefix_table"][:P // bs]
    table[:, P // bs:] = perm[shared:].view(B, tails)
    s["table"] = table
    s["pool_k"] = _pool(shared + B * tails, H, bs, d, g, torch.bfloat16)
    s["pool_v"] = _pool(shared + B * tails, H, bs, d, g, torch.bfloat16)
    s["q"] = _normal((B, Hq, d), g, torch.bfloat16)
    s["seq_lens"] = lens.to(torch.int32)
    if own:
        import top_sparse_kv_gb300 as skv

        p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=d, max_len=cap, topk=0, n_sink=0, n_local=0,
                        block_size=bs, seq_lens=s["seq_lens"])
        s["step"] = skv.PrefixStep(p, skv.Pool(s["pool_k"], s["pool_v"], s["table"]),
                                   skv.Prefix(s["prefix_table"], P))
    return s


# ---------------------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    if own:
        if case["op"] == "rope":
            q, k = s["step"].norm_rope(s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
            return dict(q=q, k=k)
        if case["op"] == "append":
            q = s["step"].append(s["q"], s["k"], s["v"], s["positions"], s["requests"], q_out=s["q_out"])
            return _appended(s, q)
        out, lse = s["step"].run(s["q"])
        return dict(out=out, lse=lse)
    if case["op"] == "rope":
        at = s["positions"]
        return dict(q=_turn(case, _norm(case, s["q"], s["gq"]), at, s["inv"]).to(s["q"].dtype),
                    k=_turn(case, _norm(case, s["k"], s["gk"]), at, s["inv"]).to(s["k"].dtype))
    if case["op"] == "append":
        return _plain_append(s)
    return _plain_prefix(s)


def _appended(s, q):
    out = dict(q=q, pool_k=s["pool_k"])
    if s["pool_v"] is not None:
        out["pool_v"] = s["pool_v"]
    return out


def _norm(case, x, gamma):
    """RMS norm of every head's leading entries, in 32 bits."""
    x = x.float()
    if gamma is None:
        return x
    n = gamma.numel()
    y = x[..., :n] * torch.rsqrt((x[..., :n] * x[..., :n]).mean(-1, keepdim=True) + 1e-6) * gamma.float()
    return y if n == x.shape[-1] else torch.cat([y, x[..., n:]], -1)


def _turn(case, x, at, inv):
    """The rotation by position; the angles in 64 bits, since far positions pass what 32 hold."""
    r, start = case["rot"], 512 if case["d"] == 576 else 0
    ang = at.double()[:, None, None] * inv.double()
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    y = x[..., start:start + r]
    if case["style"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    if r == x.shape[-1]:
        return y
    return torch.cat([x[..., :start], y, x[..., start + r:]], -1)


def _plain_append(s):
    case, at, req = s["case"], s["positions"], s["requests"]
    n = case["tokens"]
    if at is None:
        at, req = s["seq_lens"] - 1, torch.arange(n, device="cuda", dtype=torch.int32)
    keep = at >= 0
    q = _turn(case, _norm(case, s["q"], s["gq"]), at, s["inv"]).to(s["q"].dtype)
    s["q_out"][keep] = q[keep]
    k = _turn(case, _norm(case, s["k"], s["gk"]), at, s["inv"]).to(s["k"].dtype)
    at, req = at[keep].long(), req[keep].long()
    e = s["table"][req, at // s["bs"]].long()
    s["pool_k"][e, :, at % s["bs"]] = k[keep]
    if s["v"] is not None:
        s["pool_v"][e, :, at % s["bs"]] = s["v"][keep]
    return _appended(s, s["q_out"])


def _plain_prefix(s):
    case = s["case"]
    B, H, P, bs = case["batch"], case["H"], case["prefix"], BLOCK
    G, d = case["Hq"] // H, 128
    q = s["q"].float().view(B, H, G, d) * d ** -0.5
    pk = s["pool_k"][s["prefix_table"].long()].float().permute(1, 0, 2, 3).reshape(H, -1, d)[:, :P]
    pv = s["pool_v"][s["prefix_table"].long()].float().permute(1, 0, 2, 3).reshape(H, -1, d)[:, :P]
    own_blocks = s["table"][:, P // bs:].long()
    tk = s["pool_k"][own_blocks].float().permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)
    tv = s["pool_v"][own_blocks].float().permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)
    at = P // bs * bs + torch.arange(tk.shape[2], device="cuda")
    lens = s["seq_lens"].long()
    live = (at >= P) & (at < lens[:, None])
    rows = q.transpose(0, 1).reshape(H, B * G, d)
    zp = (rows @ pk.transpose(1, 2)).view(H, B, G, P)
    zt = (q @ tk.transpose(2, 3)).masked_fill(~live[:, None, None], -math.inf)
    m = torch.maximum(zp.amax(-1).transpose(0, 1), zt.amax(-1))[..., None]
    zp = torch.exp(zp.sub_(m.transpose(0, 1)))
    zt = torch.exp(zt - m)
    total = zp.sum(-1).transpose(0, 1)[..., None] + zt.sum(-1, keepdim=True)
    o = (zp.view(H, B * G, P) @ pv).view(H, B, G, d).transpose(0, 1) + zt @ tv
    on = (lens > 0)[:, None, None, None]
    out = torch.where(on, o / total, 0.0).reshape(B, H * G, d).to(torch.bfloat16)
    lse = torch.where(on, m + torch.log(total), -math.inf).reshape(B, H * G)
    return dict(out=out, lse=lse)


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    H, Hq = case["H"], case["Hq"]
    if case["op"] == "prefix":
        B, P, T = case["batch"], case["prefix"], case["tail"]
        live = B - case["empty"]
        tails = live * T / 2  # tails are uniform in 0..T
        return dict(bytes=(P + tails) * H * 128 * 2 * 2 + B * Hq * (128 * 2 * 2 + 4),
                    flops=4.0 * 128 * Hq * (live * P + tails))
    e, n, d = 4 if case["dtype"] == "f32" else 2, case["tokens"], case["d"]
    if case["op"] == "append" and not case["decode"]:
        n = n // case["batch"] * case["batch"]
    v = 2 * H * d if case["op"] == "append" and d != 576 else 0
    rows = Hq + H
    return dict(bytes=float(n) * e * (2 * rows * d + v),
                flops=float(n) * rows * (3 * case["rot"] + (4 * d if case["norm"] else 0)))


# ---------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(case, s)
    n, d, r = case["tokens"], case["d"], case["rot"]
    if s["positions"] is None:
        at, req = s["seq_lens"].long() - 1, torch.arange(n, device="cuda")
    else:
        at = s["positions"].long()
        req = None if s["requests"] is None else s["requests"].long()
    first = 512 if d == 576 else 0
    # a pair (a, b) as the complex number a + ib, turned by e^(i t f)
    turn = torch.exp(1j * (at.to(torch.float64)[:, None] * s["inv"].to(torch.float64)[None]))[:, None]
    i = torch.arange(r // 2, device="cuda")
    ia, ib = (first + i, first + i + r // 2) if case["style"] == "half" else (first + 2 * i, first + 2 * i + 1)

    def rows(x, gamma):
        x = x.to(torch.float64).clone()
        if gamma is not None:
            m = gamma.numel()
            ms = x[..., :m].pow(2).sum(-1, keepdim=True) / m
            x[..., :m] = x[..., :m] / torch.sqrt(ms + 1e-6) * gamma.to(torch.float64)
        z = torch.complex(x[..., ia], x[..., ib]) * turn
        x[..., ia], x[..., ib] = z.real, z.imag
        return x

    q, k = rows(s["q"], s["gq"]), rows(s["k"], s["gk"])
    if case["op"] == "rope":
        return dict(q=q, k=k)
    on = torch.nonzero(at >= 0).flatten()
    pk = s["pool_k"].to(torch.float64)
    t, b = at[on], req[on]
    e = s["table"].long()[b, torch.div(t, s["bs"], rounding_mode="floor")]
    off = t - torch.div(t, s["bs"], rounding_mode="floor") * s["bs"]
    pk[e, :, off] = k[on]
    q[at < 0] = 0.0
    res = dict(q=q, pool_k=pk)
    if s["v"] is not None:
        pv = s["pool_v"].to(torch.float64)
        pv[e, :, off] = s["v"][on].to(torch.float64)
        res["pool_v"] = pv
    return res


def _exact_prefix(case, s):
    B, H, P = case["batch"], case["H"], case["prefix"]
    G = case["Hq"] // H
    lens = s["seq_lens"].tolist()
    out = torch.zeros((B, H * G, 128), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for h in range(H):
        kh = s["pool_k"][s["prefix_table"].long(), h].to(torch.float64).flatten(0, 1)[:P]
        vh = s["pool_v"][s["prefix_table"].long(), h].to(torch.float64).flatten(0, 1)[:P]
        for b in range(B):
            if lens[b] == 0:
                continue
            first, last = P // BLOCK, (lens[b] + BLOCK - 1) // BLOCK
            mine = s["table"][b, first:last].long()
            lo, hi = P - first * BLOCK, lens[b] - first * BLOCK
            k = torch.cat([kh, s["pool_k"][mine, h].to(torch.float64).flatten(0, 1)[lo:hi]])
            v = torch.cat([vh, s["pool_v"][mine, h].to(torch.float64).flatten(0, 1)[lo:hi]])
            z = s["q"][b, h * G:(h + 1) * G].to(torch.float64) @ k.T / math.sqrt(128.0)
            top = z.max(-1, keepdim=True).values
            w = torch.exp(z - top)
            tot = w.sum(-1, keepdim=True)
            out[b, h * G:(h + 1) * G] = w @ v / tot
            lse[b, h * G:(h + 1) * G] = (top + torch.log(tot)).flatten()
    return dict(out=out, lse=lse)
