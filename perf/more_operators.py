"""Workloads of the operators around a KV cache held in 4 bits: the block tables and slot maps
of a step from its requests' lengths, the append of new tokens in 4 bits with the rows read
back, the scores of a whole history, and attention over a selection or over everything.
Each has its plain form (elementary torch operations in 32 bits) and, where `own` is true,
the library's calls.

A row of 128 entries is held as groups of 32, 64 or 128 with a bf16 step s and centre z each:
entry = s (c - 8) + z, c in 0..15.  Sixteen tokens of a head are one cell: their 64-byte rows of
codes, then their groups' (s, z) words.  Byte 8 i + u of a row (entries 16 i + 2 u and the
next) is stored at 8 u + i.

Sizes follow the seeded workloads of this repository (8 KV and 64 query heads of 128, 32K
histories with 3,277 selected, a history of 1,048,576) or are generic ragged ones.
"""

import math

import torch

own = False

ROPE_BASE = 500000.0
D = 128


def listed():
    return [
        # a decode step of 64 requests: a token each, now and then a new block; all latency
        dict(name="tables_step_64", op="tables", batch=64, cap=32768, new=1, even=True, base=0, bs=16),
        # prompts of 256 requests arrive at once behind a shared prefix that ends inside a block
        dict(name="tables_prompts_256", op="tables", batch=256, cap=131072, new=8192, even=False, base=1003, bs=16),
        # one new token for each of 64 requests into the cache, and back out of it
        dict(name="append_decode_64", op="append", batch=64, longest=500, decode=True, tokens=64, H=8, Hq=64,
             dtype="bf16", rot=128, style="half", norm=True, group=32, bs=16),
        # a prefill batch of 8 prompts of 1,024 through one layer
        dict(name="append_prefill_8192", op="append", batch=8, longest=4096, decode=False, tokens=8192, H=8, Hq=64,
             dtype="bf16", rot=128, style="half", norm=True, group=32, bs=16),
        # an odd count of fp32 tokens, partial rotation in pairs, groups of five heads, pages of 64, padding
        dict(name="append_odd_f32", op="append", batch=5, longest=700, decode=False, tokens=1237, H=8, Hq=40,
             dtype="f32", rot=64, style="pair", norm=True, group=64, bs=64),
        # the rows that a step attends, as a caller's own kernel takes them
        dict(name="gather_b8_32k", op="gather", batch=8, H=8, Hq=64, cap=32768, k=3277, ns=4, nl=128, group=32, bs=16,
             empty=0, full=True),
        # the selection's scan: 8 requests of 32K
        dict(name="score_b8_32k", op="score", batch=8, H=8, Hq=64, cap=32768, ns=4, nl=128, agg="mean", group=32,
             bs=16, empty=0, full=True),
        # every query head scores; ragged histories, groups of 7 heads
        dict(name="score_heads_b5", op="score", batch=5, H=4, Hq=28, cap=10007, ns=16, nl=100, agg="head", group=64,
             bs=32, empty=1, full=False),
        # four short requests: all latency
        dict(name="attn_b4_777", op="attn", batch=4, H=8, Hq=64, cap=777, k=-1, ns=0, nl=0, group=32, bs=16, empty=0,
             full=False),
        # the serving batch of 8, over everything
        dict(name="attn_b8_32k", op="attn", batch=8, H=8, Hq=64, cap=32768, k=-1, ns=0, nl=0, group=32, bs=16,
             empty=0, full=True),
        # the same batch over the selected tenth
        dict(name="attn_topk_b8_32k", op="attn", batch=8, H=8, Hq=64, cap=32768, k=3277, ns=4, nl=128, group=32,
             bs=16, empty=0, full=True),
        # one request with a million tokens of history
        dict(name="attn_b1_1m", op="attn", batch=1, H=8, Hq=32, cap=1048576, k=-1, ns=0, nl=0, group=128, bs=16,
             empty=0, full=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "gather", "score", "attn", "attn"])
    bs = rng.choice([16, 16, 32, 64])
    if op == "tables":
        batch, new = _log(rng, 1, 1000), _log(rng, 1, 8000)
        new = min(new, 1000000 // batch)
        return dict(op=op, batch=batch, cap=new + _log(rng, 100, 50000), new=new, even=rng.random() < 0.5,
                    base=rng.choice([0, 0, _log(rng, 1, 3000)]), bs=bs)
    H = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    group = rng.choice([32, 32, 64, 128])
    if op == "append":
        decode = rng.random() < 0.4
        batch = _log(rng, 1, 64) if decode else rng.randint(1, 8)
        longest = _log(rng, 20, 600) if decode else _log(rng, 20, 2000)
        return dict(op=op, batch=batch, longest=longest, decode=decode,
                    tokens=batch if decode else rng.randint(1, batch * longest), H=H, Hq=H * G,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), rot=rng.choice([32, 64, 128]),
                    style=rng.choice(["half", "pair"]), norm=rng.random() < 0.75, group=group, bs=bs)
    batch = _log(rng, 1, 64)
    cap = _log(rng, 1, max(2, min(200000, 2000000 // (batch * H))))
    case = dict(op=op, batch=batch, H=H, Hq=H * G, cap=cap, ns=rng.choice([0, 4, 16]), nl=rng.choice([0, 100, 128]),
                group=group, bs=bs, empty=rng.randint(0, batch // 8), full=rng.random() < 0.3)
    if op == "score":
        return dict(case, agg=rng.choice(["mean", "max", "head"]))
    k = _log(rng, 1, max(1, cap // 4))
    return dict(case, k=k if op == "gather" or rng.random() < 0.5 else -1)


# ---------------------------------------------------------------------------- rows in 4 bits


def _quant(x, group):
    """(codes, s, z) of [..., 128] rows: s, z bf16 [..., 128 / group], codes in 0..15.  In 64 bits: a
    value next to the border of two codes falls to the nearer one."""
    g = x.double().unflatten(-1, (D // group, group))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / 15).to(torch.bfloat16)
    z = (0.5 * (hi + lo) + 0.5 * s.double()).to(torch.bfloat16)
    c = torch.round((g - z.double()[..., None]) / s.double()[..., None])
    c = torch.where(s[..., None] == 0, 0.0, c).clamp(-8, 7) + 8
    return c.flatten(-2).to(torch.uint8), s, z


def _rows_to_cell(c, s, z):
    """The bytes of rows in order: codes [..., 64], words [..., 4 * groups]."""
    b = c[..., 0::2] | (c[..., 1::2] << 4)
    b = b.unflatten(-1, (8, 8)).transpose(-1, -2).flatten(-2)
    w = torch.stack([s, z], -1).contiguous().view(torch.uint8).flatten(-2)
    return b.contiguous(), w


def _cells(pool, group):
    """Views of a pool [n, H, bs / 16, cell]: codes [n, H, cells, 16, 64], words [n, H, cells, 16, 4 * groups]."""
    return (pool[..., :1024].unflatten(-1, (16, 64)), pool[..., 1024:].unflatten(-1, (16, 4 * (D // group))))


def _values(b, w, group):
    """fp32 rows from their bytes."""
    b = b.unflatten(-1, (8, 8)).transpose(-1, -2).flatten(-2)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    w = w.contiguous().view(torch.bfloat16).float().unflatten(-1, (D // group, 2))
    c = c.unflatten(-1, (D // group, group))
    return ((c - 8) * w[..., 0:1] + w[..., 1:2]).flatten(-2)


def _make_pool(blocks, H, bs, group, g):
    """Rows ~ N(0, 1) per channel scale, quantised; a part of the pool at a time."""
    cell = 16 * (64 + 4 * (D // group))
    pool = torch.empty((blocks, H, bs // 16, cell), dtype=torch.uint8, device="cuda")
    scale = 0.5 + torch.rand((D,), generator=g, device="cuda")
    step = max(1, (1 << 21) // (H * bs))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, H, bs // 16, 16, D), generator=g, device="cuda") * scale
        b, w = _rows_to_cell(*_quant(x, group))
        pool[i:i + n] = torch.cat([b.flatten(-2), w.flatten(-2)], -1)
    return pool


# ---------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int64)


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    return {"tables": _prepare_tables, "append": _prepare_append}.get(case["op"], _prepare_history)(case, g, s)


def _prepare_tables(case, g, s):
    B, cap, base, bs = case["batch"], case["cap"], case["base"], case["bs"]
    new = case["new"]
    cap = max(cap, base + 2 * new)
    s["cap"], per = cap, (cap + bs - 1) // bs
    # an eighth of the rows is unused; the others hold the prefix and some tokens of their own
    room = cap - new - base
    lens = base + _ints(1, room + 1, (B,), g)
    lens = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.125, 0, lens)
    n_new = torch.full((B,), new, dtype=torch.int64, device="cuda") if case["even"] else _ints(0, new + 1, (B,), g)
    s["seq_lens"], s["n_new"] = lens.to(torch.int32), n_new.to(torch.int32)
    s["n_drop"] = -s["n_new"]  # of a step whose tokens are all taken back
    s["tokens"] = B * new  # the room of the step's buffers: rows past the tokens are padding
    total = B * per
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = order.view(B, per).clone()
    first = base // bs
    have = torch.where(lens > base, (lens + bs - 1) // bs, first)
    j = torch.arange(per, device="cuda")
    taken = (j >= first) & (j < have[:, None])
    rest = table[~taken]
    s["free"] = torch.zeros((total,), dtype=torch.int32, device="cuda")
    s["free"][:rest.numel()] = rest
    s["table"] = torch.where(taken, table, -1).to(torch.int32)
    s["count"] = int(rest.numel())
    if own:
        import top_sparse_kv_gb300 as skv

        p = skv.Problem(batch=B, n_kv_heads=1, n_q_heads=1, d_qk=D, d_v=D, max_len=cap, topk=0, n_sink=0, n_local=0,
                        block_size=bs, seq_lens=s["seq_lens"])
        s["step"] = skv.BlockTables(p, s["table"], s["free"], n_free=s["count"], base=base)
    else:
        s["state"] = torch.tensor([s["count"]], dtype=torch.int32, device="cuda")
    return s


def _prepare_append(case, g, s):
    dtype, r = _dtype(case), case["rot"]
    n, H, Hq, B, cap, bs = case["tokens"], case["H"], case["Hq"], case["batch"], case["longest"], case["bs"]
    s["inv"] = (ROPE_BASE ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).to(torch.float32).cuda()
    s["gq"] = s["gk"] = None
    if case["norm"]:
        s["gk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)
        s["gq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    row = _normal((n, (Hq + 2 * H) * D), g, dtype)  # the projection's fused output
    s["q"] = row[:, :Hq * D].view(n, Hq, D)
    s["k"] = row[:, Hq * D:(Hq + H) * D].view(n, H, D)
    s["v"] = row[:, (Hq + H) * D:].view(n, H, D)
    s["q_out"] = torch.zeros((n, Hq, D), dtype=dtype, device="cuda")  # padding tokens are never written
    per = (cap + bs - 1) // bs
    s["table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    s["pool_k"] = _make_pool(B * per, H, bs, case["group"], g)
    s["pool_v"] = _make_pool(B * per, H, bs, case["group"], g)
    share = 1
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
    s["seq_lens"], s["nl"] = lens, max(share, 1)
    if own:
        import top_sparse_kv_gb300 as skv

        # the window is the new tokens, so that a gather without a selection reads them back (as bf16:
        # the attention's type, whatever the tokens' own)
        sizes = dict(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=D, d_v=D, max_len=cap, topk=0, n_sink=0,
                     n_local=s["nl"], block_size=bs, seq_lens=lens)
        p = skv.Problem(dtype=skv.SKV_DTYPE_F32 if dtype == torch.float32 else skv.SKV_DTYPE_BF16, **sizes)
        rot = skv.Rotary(inv_freq=s["inv"], rot_dim=r, style=skv.SKV_ROPE_HALF if case["style"] == "half"
                         else skv.SKV_ROPE_PAIR, norm_dim=D, eps=1e-6, q_gamma=s["gq"], k_gamma=s["gk"])
        pool = skv.Kv4Pool(s["pool_k"], s["pool_v"], s["table"], group=case["group"])
        s["tokens"], s["step"] = skv.TokenStep(p, rot, pool), skv.Kv4Step(skv.Problem(**sizes), pool)
    return s


def _prepare_history(case, g, s):
    B, H, Hq, cap, bs = case["batch"], case["H"], case["Hq"], case["cap"], case["bs"]
    lens = torch.full((B,), cap, dtype=torch.int64, device="cuda") if case["full"] else _ints(1, cap + 1, (B,), g)
    order = torch.randperm(B, generator=g, device="cuda")
    lens = torch.where(torch.isin(torch.arange(B, device="cuda"), order[:case["empty"]]), 0, lens)
    per = (cap + bs - 1) // bs
    s["seq_lens"] = lens.to(torch.int32)
    s["table"] = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    s["pool_k"] = _make_pool(B * per, H, bs, case["group"], g)
    s["pool_v"] = _make_pool(B * per, H, bs, case["group"], g) if case["op"] != "score" else s["pool_k"]
    s["q"] = _normal((B, Hq, D), g, torch.bfloat16)
    k = case.get("k", -1)
    s["idx"] = None
    if k > 0:
        # a selection among the candidates, ascending, -1 past the end of short ones
        lo, hi = _regions(case, lens)
        t = torch.arange(cap, device="cuda")
        live = (t >= lo[:, None]) & (t < hi[:, None])
        key = torch.rand((B, H, cap), generator=g, device="cuda").masked_fill_(~live[:, None], -1.0)
        top = key.topk(min(k, cap), -1)
        at = torch.where(top.values >= 0, top.indices, cap).sort(-1).values
        s["idx"] = torch.full((B, H, k), -1, dtype=torch.int32, device="cuda")
        s["idx"][..., :at.shape[-1]] = torch.where(at < cap, at, -1).to(torch.int32)
    if case["op"] == "score":
        # (a row is written over the candidates of its request; the rest stays)
        s["scores"] = torch.zeros((B, Hq if case["agg"] == "head" else H, cap), device="cuda")
    if own:
        import top_sparse_kv_gb300 as skv

        agg = {"mean": skv.SKV_AGG_MEAN, "max": skv.SKV_AGG_MAX, "head": skv.SKV_AGG_HEAD}[case.get("agg", "mean")]
        p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=D, d_v=D, max_len=cap, topk=max(k, 0),
                        n_sink=case["ns"], n_local=case["nl"], block_size=bs, seq_lens=s["seq_lens"], group_agg=agg)
        s["step"] = skv.Kv4Step(p, skv.Kv4Pool(s["pool_k"], s["pool_v"], s["table"], group=case["group"]))
    return s


def _regions(case, lens):
    """Candidates [lo, hi) of each request: what is in neither the sink nor the window."""
    lo = lens.clamp(max=case["ns"])
    return lo, torch.maximum(lo, lens - case["nl"])


# ---------------------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "tables":
        return _run_tables(s)
    if own:
        if op == "append":
            q = s["tokens"].append(s["q"], s["k"], s["v"], s["positions"], s["requests"], q_out=s["q_out"])
            k, v = s["step"].gather()
            return dict(q=q, k=k, v=v)
        if op == "gather":
            k, v = s["step"].gather(s["idx"])
            return dict(k=k, v=v)
        if op == "score":
            return dict(scores=s["step"].score(s["q"], s["scores"]))
        out, lse = s["step"].attend(s["q"], s["idx"]) if s["idx"] is not None else s["step"].attend_all(s["q"])
        return dict(out=out, lse=lse)
    return {"append": _plain_append, "gather": _plain_gather, "score": _plain_score, "attn": _plain_attn}[op](s)


def _run_tables(s):
    if own:
        at, req, slots = s["step"].update(s["n_new"], s["tokens"])
        s["step"].update(s["n_drop"])
        count = s["step"].n_free
    else:
        at, req, slots = _plain_tables(s, s["n_new"], s["tokens"])
        _plain_tables(s, s["n_drop"], 0)
        count = s["state"]
    return dict(positions=at, requests=req, slots=slots, table=s["table"], seq_lens=s["seq_lens"], free=s["free"],
                count=count)


def _plain_tables(s, n_new, tokens):
    """Every request takes n_new more tokens (or gives the last -n_new back): its length, its
    blocks off (or back onto) the stack of free ones, and each token's position, request and row."""
    case = s["case"]
    B, base, bs, cap = case["batch"], case["base"], case["bs"], s["cap"]
    old, n, count = s["seq_lens"].long(), n_new.long(), s["state"].long()
    start = torch.where(old == 0, base, old)
    grow, drop = n > 0, n < 0
    have = torch.where(old > base, (old + bs - 1) // bs, base // bs)
    upto = start + n
    tok = torch.where(grow, n, 0).cumsum(0)
    need = torch.where(grow & (upto <= cap), (upto + bs - 1) // bs - have, 0)
    cum = need.cumsum(0)
    ok = grow & (upto <= cap) & (tok <= tokens) & ((need == 0) | (cum <= count))
    left = torch.where(drop, torch.where(old + n > base, old + n, 0), old)
    keep = torch.where(left > base, (left + bs - 1) // bs, base // bs)
    gone = torch.where(drop, have - keep, 0)
    # the blocks given back, the last request's last first, go onto the stack in that order
    cg = gone.flip(0).cumsum(0)
    back = torch.arange(s["table"].shape[1], device="cuda")
    mask = drop[:, None] & (back >= keep[:, None]) & (back < have[:, None])
    freed = s["table"].flip(0, 1)[mask.flip(0, 1)]
    s["free"][int(count):int(count) + freed.numel()] = freed
    # blocks taken off its top, in the requests' order
    got = torch.where(ok, need, 0)
    mask = (back >= have[:, None]) & (back < (have + got)[:, None])
    total = int(got.sum())
    s["table"][mask] = s["free"][:int(count)].flip(0)[:total]
    s["state"].copy_(count - total + cg[-1:])
    s["seq_lens"].copy_(torch.where(ok, upto, left))
    i = torch.arange(tokens, device="cuda")
    req = torch.searchsorted(tok, i, right=True)
    real = req < B
    req = req.clamp(max=B - 1)
    real &= ok[req]
    at = start[req] + i - (tok - torch.where(grow, n, 0))[req]
    e = s["table"][req, torch.where(real, at, 0) // bs].long()
    none = torch.full_like(i, -1)
    return (torch.where(real, at, none).to(torch.int32), torch.where(real, req, none).to(torch.int32),
            torch.where(real, e * bs + at % bs, none))


def _norm(x, gamma, bits=torch.float32):
    x = x.to(bits)
    if gamma is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma.to(bits)


def _turn(case, x, at, inv):
    """The rotation by position; the angles in 64 bits, since far positions pass what 32 hold."""
    r = case["rot"]
    ang = at.double()[:, None, None] * inv.double()
    c, s = torch.cos(ang).to(x.dtype), torch.sin(ang).to(x.dtype)
    y = x[..., :r]
    if case["style"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return y if r == D else torch.cat([y, x[..., r:]], -1)


def _plain_append(s):
    case, at, req = s["case"], s["positions"], s["requests"]
    n, group, bs = case["tokens"], case["group"], case["bs"]
    if at is None:
        at, req = s["seq_lens"] - 1, torch.arange(n, device="cuda", dtype=torch.int32)
    keep = at >= 0
    q = _turn(case, _norm(s["q"], s["gq"]), at, s["inv"]).to(s["q"].dtype)
    s["q_out"][keep] = q[keep]
    k = _turn(case, _norm(s["k"], s["gk"], torch.float64), at, s["inv"])  # (see _quant)
    at, req = at[keep].long(), req[keep].long()
    e, off = s["table"][req, at // bs].long(), at % bs
    for pool, x in ((s["pool_k"], k), (s["pool_v"], s["v"])):
        b, w = _rows_to_cell(*_quant(x[keep], group))
        codes, words = _cells(pool, group)
        codes[e, :, off // 16, off % 16] = b
        words[e, :, off // 16, off % 16] = w
    return dict(q=s["q_out"], **_read(s, _attended(s, 0, s["nl"], None), torch.bfloat16))


def _attended(s, ns, nl, idx):
    """Positions [B, H, n_att] that a step attends: sink, selection, window; -1 where there is none."""
    lens = s["seq_lens"].long()[:, None, None]
    k = 0 if idx is None else idx.shape[-1]
    j = torch.arange(ns + k + nl, device="cuda")
    end = lens.clamp(max=ns)
    first = torch.maximum(end, lens - nl)
    at = torch.where(j < end, j, torch.where(j < end + k + lens - first, first + j - end - k, -1))
    at = at.expand(-1, s["case"]["H"], -1)
    if k:
        sel = torch.gather(idx.long(), -1, (j - end).clamp(0, k - 1).expand(at.shape))
        at = torch.where((j >= end) & (j < end + k), sel, at)
    return at


def _row_bytes(pool, s, at, group):
    bs, H = s["case"]["bs"], s["case"]["H"]
    t = at.clamp(min=0)
    b = torch.arange(at.shape[0], device="cuda")[:, None, None]
    h = torch.arange(H, device="cuda")[:, None]
    e = s["table"][b, t // bs].long()
    codes, words = _cells(pool, group)
    off = t % bs
    return codes[e, h, off // 16, off % 16], words[e, h, off // 16, off % 16]


def _read(s, at, dtype):
    group = s["case"]["group"]
    on = (at >= 0)[..., None]
    k, v = (torch.where(on, _values(*_row_bytes(p, s, at, group), group), 0.0) for p in (s["pool_k"], s["pool_v"]))
    return dict(k=k.to(dtype), v=v.to(dtype))


def _plain_gather(s):
    case = s["case"]
    return _read(s, _attended(s, case["ns"], case["nl"], s["idx"]), torch.bfloat16)


def _history(pool, s, b):
    """Every row of request b: fp32 [H, per * bs, 128]."""
    group = s["case"]["group"]
    codes, words = _cells(pool[s["table"][b].long()], group)
    return _values(codes, words, group).permute(1, 0, 2, 3, 4).flatten(1, 3)


def _plain_score(s):
    case = s["case"]
    H, cap = case["H"], case["cap"]
    lens = s["seq_lens"].long()
    lo, hi = _regions(case, lens)
    t = torch.arange(cap, device="cuda")
    for b in range(case["batch"]):
        q = s["q"][b].float().view(H, -1, D)
        k = _history(s["pool_k"], s, b)[:, :cap].transpose(1, 2)
        if case["agg"] == "mean":
            z = q.mean(1, keepdim=True) @ k
        else:
            z = q @ k
            if case["agg"] == "max":
                z = z.amax(1, keepdim=True)
        on = (t >= lo[b]) & (t < hi[b])
        s["scores"][b] = torch.where(on, z.flatten(0, 1), s["scores"][b])
    return dict(scores=s["scores"])


def _plain_attn(s):
    case = s["case"]
    B, H, Hq = case["batch"], case["H"], case["Hq"]
    lens = s["seq_lens"].long()
    out = torch.empty((B, H, Hq // H, D), device="cuda")
    lse = torch.empty((B, H, Hq // H), device="cuda")
    at = None if s["idx"] is None else _attended(s, case["ns"], case["nl"], s["idx"])
    t = torch.arange(s["table"].shape[1] * case["bs"], device="cuda")
    for b in range(B):
        q = s["q"][b].float().view(H, -1, D) * D ** -0.5
        if at is None:
            k, v, on = _history(s["pool_k"], s, b), _history(s["pool_v"], s, b), (t < lens[b]).expand(H, -1)
        else:
            one = dict(s, table=s["table"][b:b + 1])
            rows = [_values(*_row_bytes(p, one, at[b:b + 1], case["group"]), case["group"])[0]
                    for p in (s["pool_k"], s["pool_v"])]
            k, v, on = rows[0], rows[1], at[b] >= 0
        z = (q @ k.transpose(1, 2)).masked_fill(~on[:, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        o = (p @ v) / total
        out[b] = torch.where(total > 0, o, 0.0)
        lse[b] = (m + torch.log(total))[..., 0]
    return dict(out=out.view(B, Hq, D).to(torch.bfloat16), lse=lse.view(B, Hq))


# ---------------------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "tables":
        B, new, bs = case["batch"], case["new"], case["bs"]
        tokens = B * new * (1.0 if case["even"] else 0.5)
        blocks = tokens / bs
        # the maps, the tables' new entries, the stack's both ways; lengths and counts of two calls
        return dict(bytes=16.0 * B * new + 16.0 * blocks + 24.0 * B, flops=10.0 * tokens)
    H, Hq, row = case["H"], case["Hq"], 64 + 4 * (D // case["group"])
    if op == "append":
        e, n = 4 if case["dtype"] == "f32" else 2, case["tokens"]
        if not case["decode"]:
            n = n // case["batch"] * case["batch"]
        return dict(bytes=float(n) * (e * D * (2 * Hq + 2 * H) + 2 * H * row + 2 * H * (row + 2 * D)),
                    flops=float(n) * ((Hq + H) * (3 * case["rot"] + (4 * D if case["norm"] else 0)) + 12 * D * H))
    B, cap = case["batch"], case["cap"]
    live = (B - case["empty"]) * (cap if case["full"] else cap / 2)
    att = (B - case["empty"]) * min(cap if case["full"] else cap / 2, case["ns"] + case["nl"] + max(case.get("k", 0), 0))
    if op == "score":
        rows = Hq if case["agg"] == "head" else H
        return dict(bytes=live * (H * row + 4.0 * rows) + B * Hq * D * 2,
                    flops=2.0 * D * live * (H if case["agg"] == "mean" else Hq))
    if op == "gather":
        return dict(bytes=2.0 * H * (att * row + B * (case["ns"] + case["k"] + case["nl"]) * 2 * D) + 4.0 * B * H * case["k"],
                    flops=4.0 * D * H * att)
    n = live if case["k"] < 0 else att
    return dict(bytes=2.0 * H * n * row + B * Hq * (4.0 * D + 4) + 4.0 * B * H * max(case["k"], 0),
                flops=4.0 * D * Hq * n)


# ---------------------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "gather": _exact_gather, "score": _exact_score,
            "attn": _exact_attn}[case["op"]](case, s)


def _exact_tables(case, s):
    """One request at a time, blocks by a Python list; the drop undoes it, so lengths and stack are the old ones."""
    bs, base, T = case["bs"], case["base"], s["tokens"]
    lens, news = s["seq_lens"].tolist(), s["n_new"].tolist()
    stack = s["free"][:s["count"]].tolist()
    table = s["table"].cpu()
    at = torch.full((T,), -1, dtype=torch.int32)
    req, slots = at.clone(), torch.full((T,), -1, dtype=torch.int64)
    row = 0
    for b, (length, n) in enumerate(zip(lens, news)):
        if n <= 0:
            continue
        first = length if length else base
        have = -(-length // bs) if length > base else base // bs
        for j in range(have, -(-(first + n) // bs)):
            table[b, j] = stack.pop()
        t = torch.arange(first, first + n)
        at[row:row + n], req[row:row + n] = t.to(torch.int32), b
        slots[row:row + n] = table[b, t // bs].long() * bs + t % bs
        row += n
    return dict(positions=at.cuda(), requests=req.cuda(), slots=slots.cuda(), table=table.cuda(),
                seq_lens=s["seq_lens"].clone(), free=s["free"].clone(),
                count=torch.tensor([s["count"]], dtype=torch.int32, device="cuda"))


def _exact_rows(pool, e, h, off, group):
    """fp64 rows at block e, head h, offset off (index tensors of one shape), entry by entry."""
    j = torch.arange(D, device="cuda")
    byte = (j // 2) % 8 * 8 + j // 16
    cell, r = (off // 16)[..., None], (off % 16)[..., None]
    e, h = e[..., None], h[..., None]
    b = pool[e, h, cell, r * 64 + byte].to(torch.int64)
    c = torch.where(j % 2 == 0, b % 16, torch.div(b, 16, rounding_mode="floor"))
    w = 1024 + (r * (D // group) + j // group) * 4

    def half(at):  # two bytes, low first, the upper half of an fp32
        u = pool[e, h, cell, at].to(torch.int32) | (pool[e, h, cell, at + 1].to(torch.int32) << 8)
        return (u << 16).view(torch.float32).to(torch.float64)

    return half(w) * (c - 8).to(torch.float64) + half(w + 2)


def _exact_read(case, s, at):
    at = at.to(torch.int64)
    keep = at >= 0
    t = torch.where(keep, at, 0)
    b = torch.arange(at.shape[0], device="cuda")[:, None, None].expand_as(t)
    h = torch.arange(at.shape[1], device="cuda")[None, :, None].expand_as(t)
    e = s["table"].long()[b, torch.div(t, case["bs"], rounding_mode="floor")]
    return [_exact_rows(p, e, h, t % case["bs"], case["group"]) * keep[..., None] for p in (s["pool_k"], s["pool_v"])]


def _exact_list(case, s, ns, nl, idx):
    """The attended positions of each request, from Python's own ranges."""
    k = 0 if idx is None else idx.shape[-1]
    res = torch.full((case["batch"], case["H"], ns + k + nl), -1, dtype=torch.int64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        sink = min(n, ns)
        local = range(max(sink, n - nl), n)
        res[b, :, :sink] = torch.arange(sink, device="cuda")
        if k:
            res[b, :, sink:sink + k] = idx[b].long()
        res[b, :, sink + k:sink + k + len(local)] = torch.arange(local.start, n, device="cuda")
    return res


def _exact_append(case, s):
    n, r, group = case["tokens"], case["rot"], case["group"]
    if s["positions"] is None:
        at, req = s["seq_lens"].long() - 1, torch.arange(n, device="cuda")
    else:
        at, req = s["positions"].long(), s["requests"].long()
    # a pair (a, b) as the complex number a + ib, turned by e^(i t f)
    turn = torch.exp(1j * (at.to(torch.float64)[:, None] * s["inv"].to(torch.float64)[None]))[:, None]
    i = torch.arange(r // 2, device="cuda")
    ia, ib = (i, i + r // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)

    def rows(x, gamma):
        x = x.to(torch.float64).clone()
        if gamma is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * gamma.to(torch.float64)
        z = torch.complex(x[..., ia], x[..., ib]) * turn
        x[..., ia], x[..., ib] = z.real, z.imag
        return x

    def held(x):  # what 4 bits keep of it
        y = torch.empty_like(x)
        for lo in range(0, D, group):
            part = x[..., lo:lo + group]
            least, most = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
            step = ((most - least) / 15.0).to(torch.bfloat16).to(torch.float64)
            mid = ((most + least + step) / 2.0).to(torch.bfloat16).to(torch.float64)
            c = torch.where(step > 0, torch.round((part - mid) / step.clamp(min=1e-300)), torch.zeros_like(part))
            y[..., lo:lo + group] = step * c.clamp(-8, 7) + mid
        return y

    q = rows(s["q"], s["gq"])
    q[at < 0] = 0.0
    # the window of request b is its last nl tokens: rows of this call where they are, else the cache's
    at_back = _exact_list(case, s, 0, s["nl"], None)
    k, v = _exact_read(case, s, at_back)
    on = torch.nonzero(at >= 0).flatten()
    lens = s["seq_lens"].long()
    j = at[on] - (lens[req[on]] - s["nl"]).clamp(min=0)
    k[req[on], :, j] = held(rows(s["k"], s["gk"]))[on]
    v[req[on], :, j] = held(s["v"].to(torch.float64))[on]
    return dict(q=q, k=k, v=v)


def _exact_gather(case, s):
    k, v = _exact_read(case, s, _exact_list(case, s, case["ns"], case["nl"], s["idx"]))
    return dict(k=k, v=v)


def _exact_unit(case, s, pool, b, h, n):
    t = torch.arange(n, device="cuda")
    e = s["table"][b].long()[torch.div(t, case["bs"], rounding_mode="floor")]
    return _exact_rows(pool, e, torch.full_like(t, h), t % case["bs"], case["group"])


def _exact_score(case, s):
    H, G = case["H"], case["Hq"] // case["H"]
    res = s["scores"].to(torch.float64)
    for b, n in enumerate(s["seq_lens"].tolist()):
        lo = min(n, case["ns"])
        hi = max(lo, n - case["nl"])
        for h in range(H):
            k = _exact_unit(case, s, s["pool_k"], b, h, n)[lo:hi]
            q = s["q"][b, h * G:(h + 1) * G].to(torch.float64)
            if case["agg"] == "head":
                res[b, h * G:(h + 1) * G, lo:hi] = q @ k.T
            elif case["agg"] == "max" and hi > lo:
                res[b, h, lo:hi] = (q @ k.T).max(0).values
            elif case["agg"] == "mean":
                res[b, h, lo:hi] = k @ (q.sum(0) / G)
    return dict(scores=res)


def _exact_attn(case, s):
    B, H, G = case["batch"], case["H"], case["Hq"] // case["H"]
    out = torch.zeros((B, H * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H * G), -math.inf, dtype=torch.float64, device="cuda")
    lists = None if s["idx"] is None else _exact_list(case, s, case["ns"], case["nl"], s["idx"])
    for b, n in enumerate(s["seq_lens"].tolist()):
        for h in range(H):
            if lists is None:
                k, v = (_exact_unit(case, s, p, b, h, n) for p in (s["pool_k"], s["pool_v"]))
            else:
                t = lists[b, h][lists[b, h] >= 0]
                e = s["table"][b].long()[torch.div(t, case["bs"], rounding_mode="floor")]
                k, v = (_exact_rows(p, e, torch.full_like(t, h), t % case["bs"], case["group"])
                        for p in (s["pool_k"], s["pool_v"]))
            if k.shape[0] == 0:
                continue
            z = s["q"][b, h * G:(h + 1) * G].to(torch.float64) @ k.T / math.sqrt(D)
            top = z.max(-1, keepdim=True).values
            w = torch.exp(z - top)
            tot = w.sum(-1, keepdim=True)
            out[b, h * G:(h + 1) * G] = w @ v / tot
            lse[b, h * G:(h + 1) * G] = (top + torch.log(tot)).flatten()
    return dict(out=out, lse=lse)
