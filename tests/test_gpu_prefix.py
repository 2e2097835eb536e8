"""Attention over a shared prefix and the requests' own tails, against fp64.

Every pool starts as NaN and holds numbers in the attended rows alone, so a row read past a
history's or the prefix's end, or through another entry, shows.

Tolerance, from the arithmetic, with w the softmax weights and A = sum w |v|:
  a logit is an fp32 sum of 128 products, off by at most dz = 130 * 2^-24 * s * sum |q k|
  (the largest over the keys), and the same for every weight twice (weight and sum);
  a weight is rounded to bf16 before it meets V: 2^-8 of it; ex2 is within 2^-22;
  fp32 accumulation over n keys: at most (n / 8 + 64) roundings;
  the output's own rounding: 2^-8 of it.
"""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


class Case:
    """A batch on the GPU: pools of NaN with the attended rows filled through random tables."""

    def __init__(self, skv, B, H, G, P, lens, bs=16, host=0.0, seed=0, cap=None, first_block=0, k_scale=None,
                 own_prefix_rows=False):
        g = torch.Generator()
        g.manual_seed(seed)
        self.B, self.H, self.G, self.P, self.lens, self.bs = B, H, G, P, list(lens), bs
        cap = cap if cap is not None else max([P] + self.lens + [1])
        per, shared = (cap + bs - 1) // bs, (P + bs - 1) // bs
        n = shared + B * per
        perm = torch.randperm(n, generator=g).to(torch.int32)
        ent = perm + first_block
        on_host = torch.rand(n, generator=g) < host
        self.ptable, table = ent[:shared].clone(), ent[shared:].view(B, per).clone()
        nb = n + first_block
        nan = lambda: torch.full((nb, H, bs, D), float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if first_block:  # a long cache: only its last blocks are touched
            nan = lambda: torch.empty((nb, H, bs, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        gk, gv = nan(), nan()
        gk[first_block:], gv[first_block:] = float("nan"), float("nan")
        hk = hv = None
        if host:
            hk, hv = (torch.full((nb, H, bs, D), float("nan"), dtype=torch.bfloat16).pin_memory() for _ in range(2))
            self.ptable = torch.where(on_host[:shared], -self.ptable - 1, self.ptable)
            table = torch.where(on_host[shared:].view(B, per), -table - 1, table)
        self.keys, self.vals = [], []  # per request [L, H, D]

        def put(entries, lo, hi, x, pools):
            for blk in range(lo // bs, (hi + bs - 1) // bs):
                a, z = max(lo, blk * bs), min(hi, (blk + 1) * bs)
                e = int(entries[blk])
                pool = pools[0] if e >= 0 else pools[1]
                pool[e if e >= 0 else -e - 1, :, a - blk * bs:z - blk * bs] = x[a - lo:z - lo].transpose(0, 1).to(
                    pool.device)

        def rows(lo, hi):
            k = torch.randn((hi - lo, H, D), generator=g)
            if k_scale is not None:
                k = k * k_scale(torch.arange(lo, hi))[:, None, None]
            return k.to(torch.bfloat16), torch.randn((hi - lo, H, D), generator=g).to(torch.bfloat16)

        pk, pv = rows(0, P)
        put(self.ptable, 0, P, pk, (gk, hk)), put(self.ptable, 0, P, pv, (gv, hv))
        for b, L in enumerate(self.lens):
            if L < P or L == 0:
                self.keys.append(None), self.vals.append(None)
                continue
            k, v = rows(P, L)
            put(table[b], P, L, k, (gk, hk)), put(table[b], P, L, v, (gv, hv))
            self.keys.append(torch.cat([pk, k])), self.vals.append(torch.cat([pv, v]))
        if own_prefix_rows:  # the table's prefix entries name the shared blocks, as a paged server keeps it
            table[:, :P // bs] = self.ptable[:P // bs]
        else:  # never read: entries that no pool has
            table[:, :P // bs] = 2 ** 31 - 1
        self.q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=cap, topk=0, n_sink=0,
                             n_local=0, block_size=bs, seq_lens=self.seq_lens)
        self.pool = skv.Pool(gk, gv, table.cuda().contiguous(), hk, hv)
        self.prefix = skv.Prefix(self.ptable.cuda() if P else None, P)
        self.qd = self.q.cuda()

    def check(self, out, lse, q=None):
        q = (self.q if q is None else q).double().cuda()
        s = D ** -0.5
        worst = 0.0
        for b in range(self.B):
            got, gl = out[b].double(), lse[b].double()
            if self.keys[b] is None:
                assert torch.count_nonzero(out[b]) == 0 and bool((lse[b] == -math.inf).all()), b
                continue
            k, v = self.keys[b].cuda().double().transpose(0, 1), self.vals[b].cuda().double().transpose(0, 1)
            qb = q[b].view(self.H, self.G, D)
            z = qb @ k.transpose(1, 2) * s
            dz = 130 * 2.0 ** -24 * s * (qb.abs() @ k.abs().transpose(1, 2)).amax(-1)
            w = torch.softmax(z, -1)
            ref, A = w @ v, w @ v.abs()
            n = k.shape[1]
            tol = 2.0 ** -8 * (A + ref.abs()) + A * (2 * dz[..., None] + (n / 8 + 64) * 2.0 ** -24 + 2.0 ** -20)
            err = (got.view(self.H, self.G, D) - ref).abs()
            assert bool((err <= tol).all()), (b, float((err - tol).max()), float(err.max()))
            rl = torch.logsumexp(z, -1)
            tl = dz + (n / 128 + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * rl.abs()
            assert bool(((gl.view(self.H, self.G) - rl).abs() <= tl).all()), b
            worst = max(worst, float((err / tol).max()))
        return worst


def _tails(B, P, longest, seed, empty=0):
    g = np.random.default_rng(seed)
    lens = [P + int(x) for x in g.integers(0, longest + 1, B)]
    for i in range(empty):
        lens[(3 * i + 1) % B] = 0
    return lens


CASES = [
    # B, H, G, P, lens, kwargs
    (1, 1, 1, 1, [1], {}),
    (1, 1, 8, 1, [2], {}),
    (1, 1, 8, 128, [128], {}),
    (1, 2, 4, 129, [130], {}),
    (1, 1, 8, 0, [1], {}),
    (2, 2, 8, 0, [300, 17], {}),
    (3, 2, 5, 130, [130, 257, 259], {}),
    (4, 8, 8, 777, _tails(4, 777, 90, 1), {}),
    (5, 2, 3, 64, [0, 64, 0, 80, 0], {}),
    (3, 2, 8, 100, [0, 0, 0], {}),
    (16, 2, 8, 1000, _tails(16, 1000, 300, 2), {}),                 # 128 rows: one full tile
    (43, 1, 3, 500, _tails(43, 500, 40, 3, 3), {}),                 # 129 rows: a second tile of one row
    (32, 2, 8, 2049, _tails(32, 2049, 200, 4, 2), {}),              # 256 rows: one pair
    (60, 2, 5, 333, _tails(60, 333, 150, 5), {}),                   # 300 rows: a pair and a single
    (130, 2, 8, 700, _tails(130, 700, 140, 6, 9), {}),              # 1,040 rows: groups of pairs, one short
    (200, 1, 16, 260, _tails(200, 260, 30, 7), {}),                 # 3,200 rows
    (2, 1, 128, 300, [300, 600], {}),                               # 128 query heads on one KV head
    (7, 3, 7, 1111, _tails(7, 1111, 64, 8), dict(bs=1)),
    (5, 2, 4, 97, _tails(5, 97, 50, 9), dict(bs=7)),
    (4, 2, 4, 200, _tails(4, 200, 300, 10), dict(bs=256)),
    (20, 2, 8, 3000, _tails(20, 3000, 700, 21, 2), dict(bs=8)),
    (40, 2, 8, 1500, _tails(40, 1500, 300, 22, 2), dict(bs=24, host=0.5)),
    (40, 2, 8, 1500, _tails(40, 1500, 300, 23, 2), dict(bs=48, host=0.5)),
    (6, 2, 8, 500, _tails(6, 500, 200, 11), dict(host=0.4)),
    (6, 2, 8, 500, _tails(6, 500, 200, 12), dict(host=1.0)),
    (6, 2, 8, 512, _tails(6, 512, 200, 13), dict(own_prefix_rows=True)),
    (2, 4, 8, 40, [5000, 9000], {}),                                # long tails, a short prefix
    (8, 8, 8, 20000, _tails(8, 20000, 500, 14), {}),
    (700, 4, 2, 130, _tails(700, 130, 600, 15, 40), {}),            # some twenty short segments a CTA
    (400, 3, 2, 0, _tails(400, 0, 300, 16, 30), {}),                # no prefix at all
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_fp64(skv, case):
    B, H, G, P, lens, kw = CASES[case]
    c = Case(skv, B, H, G, P, lens, seed=case, **kw)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    out, lse = step.run(c.qd)
    c.check(out, lse)
    assert int(step.status.item()) == 0
    first = out.clone(), lse.clone()
    for _ in range(3):  # deterministic, whatever the workspace holds
        step.ws.fill_(255)
        out, lse = step.run(c.qd)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # without lse and status, through the plain binding
    o2 = torch.empty_like(out)
    skv.skv_prefix_attn(c.p, c.qd, c.pool, c.prefix, o2, None, step.ws)
    assert torch.equal(o2, first[0])


@pytest.mark.parametrize("seed", range(24))
def test_any_shape(skv, seed):
    """Batches of every kind: how the prefix's and the tails' tiles are cut over the CTAs, which
    CTAs hold a unit's partials, single and paired row tiles, gangs."""
    g = np.random.default_rng(1000 + seed)
    H, G = int(g.choice([1, 2, 3, 4, 8])), int(g.choice([1, 2, 3, 5, 8, 16]))
    B = int(np.exp(g.uniform(0, math.log(max(2, min(160, 2048 // G))))))
    P = int(np.exp(g.uniform(0, math.log(12000)))) if seed % 6 else 0
    longest = int(np.exp(g.uniform(0, math.log(1500))))
    c = Case(skv, B, H, G, P, _tails(B, P, longest, 2000 + seed, empty=int(g.integers(0, B // 4 + 1))), seed=seed)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    step.ws.fill_(255)  # NaN in every partial that is not written
    out, lse = step.run(c.qd)
    c.check(out, lse)
    assert int(step.status.item()) == 0


@pytest.mark.parametrize("shape", ["up", "down", "spikes"])
def test_running_maximum(skv, shape):
    """Keys whose size grows, falls or jumps along the history: the maximum is renewed (or must
    not be) many times, with logits of some hundreds."""
    scale = {"up": lambda t: 0.05 + 40.0 * t / 3000, "down": lambda t: 40.0 - 39.9 * (t / 3000).clamp(max=1),
             "spikes": lambda t: torch.where(t % 517 == 300, 60.0, 0.2)}[shape]
    c = Case(skv, 20, 2, 8, 2300, _tails(20, 2300, 600, 3, 1), seed=5, k_scale=scale)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    c.check(*step.run(c.qd))


def test_sm_scale(skv):
    c = Case(skv, 3, 2, 4, 200, [200, 260, 0], seed=6)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    out, lse = (t.clone() for t in step.run(c.qd))
    c.p.sm_scale = 2 * D ** -0.5
    half = skv.PrefixStep(c.p, c.pool, c.prefix)
    o2, l2 = half.run(c.qd / 2)  # powers of two: the same logits
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_lengths_inside_the_prefix_and_outside_the_table(skv):
    c = Case(skv, 5, 2, 4, 300, [300, 299, 1, 340, 350], seed=7, cap=350)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    out, lse = step.run(c.qd)
    c.check(out, lse)  # requests 1 and 2 end inside the prefix: out 0, lse -inf
    assert int(step.status.item()) == skv.SKV_DEV_BAD_LENGTH
    full = out[4].clone()
    step.status.zero_()
    c.seq_lens.copy_(torch.tensor([300, 0, -5, 340, 1000], dtype=torch.int32))
    out, lse = step.run(c.qd)  # past the capacity: clamped to it
    assert torch.equal(out[4], full)
    c.check(out, lse)
    assert int(step.status.item()) == skv.SKV_DEV_BAD_LENGTH


def test_bad_entries_get_no_weight(skv):
    c = Case(skv, 3, 2, 4, 100, [100, 150, 260], seed=8)
    c.ptable[2] = c.pool.gpu_k.shape[0]            # positions 32..47: past the GPU pool
    c.pool.slot_table[2, 10] = -1                  # positions 160..175: no host pool
    px = skv.Prefix(c.ptable.cuda(), 100)
    step = skv.PrefixStep(c.p, c.pool, px)
    out, lse = step.run(c.qd)
    for b in range(3):
        keep = torch.ones(c.keys[b].shape[0], dtype=torch.bool)
        keep[32:48] = False
        if b == 2:
            keep[160:176] = False
        c.keys[b], c.vals[b] = c.keys[b][keep], c.vals[b][keep]
    c.check(out, lse)
    assert int(step.status.item()) == skv.SKV_DEV_BAD_SLOT
    # every entry bad: rows without a key
    step = skv.PrefixStep(c.p, c.pool, skv.Prefix(torch.full_like(px.table, 2 ** 31 - 1), 100))
    out, lse = step.run(c.qd)
    assert torch.count_nonzero(out[0]) == 0 and bool((lse[0] == -math.inf).all())


def test_nonfinite_queries_and_keys_stay_in_their_rows(skv):
    c = Case(skv, 20, 2, 8, 400, _tails(20, 400, 100, 9), seed=9)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    clean = step.run(c.qd)[0].clone()
    q = c.q.clone()
    q[3, 5, 7], q[19, 15, 0] = float("nan"), float("inf")
    out, _ = step.run(q.cuda())
    hit = torch.zeros(20, 16, dtype=torch.bool)
    hit[3, 5] = hit[19, 15] = True
    assert bool(torch.isnan(out[3, 5]).all())
    assert torch.equal(out[~hit], clean[~hit])


def test_offsets_past_32_bits(skv):
    """Blocks past 4 GB of the pool (and past 2^31 elements)."""
    first = 140_000  # of 32 KB each
    c = Case(skv, 4, 8, 4, 333, _tails(4, 333, 60, 10), seed=10, first_block=first)
    assert (c.pool.gpu_k.numel() >> 31) >= 1
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    c.check(*step.run(c.qd))


def test_millions_of_keys(skv):
    """So many tail tiles that their cut is counted in 64 bits: one request's 5,000,000 positions all
    name one block, so it attends that block's 16 keys 312,500 times; others have a few keys."""
    H, n = 16, 5_000_000
    c = Case(skv, 3, H, 1, 0, [200, 100, 0], seed=19, cap=208)
    per = n // 16
    table = torch.full((3, per), 2 ** 31 - 1, dtype=torch.int32)
    table[:, :13] = c.pool.slot_table.cpu()
    table[0] = table[0, 0]
    k, v = c.keys[0][:16], c.vals[0][:16]
    lens = torch.tensor([n, 100, 0], dtype=torch.int32).cuda()
    p = skv.Problem(batch=3, n_kv_heads=H, n_q_heads=H, d_qk=D, d_v=D, max_len=n, topk=0, n_sink=0, n_local=0,
                    block_size=16, seq_lens=lens)
    step = skv.PrefixStep(p, skv.Pool(c.pool.gpu_k, c.pool.gpu_v, table.cuda()), skv.Prefix(None, 0))
    step.ws.fill_(255)
    out, lse = step.run(c.qd)
    assert int(step.status.item()) == 0
    q = c.q[0].double().view(H, 1, D)
    kd, vd = k.double().transpose(0, 1), v.double().transpose(0, 1)
    z = (q @ kd.transpose(1, 2) * D ** -0.5)[:, 0]
    w = torch.softmax(z, -1)[:, None]
    ref, A = (w @ vd)[:, 0], (w @ vd.abs())[:, 0]
    dz = 130 * 2.0 ** -24 * D ** -0.5 * (q.abs() @ kd.abs().transpose(1, 2)).amax(-1)
    # a CTA's slot adds up to 2,100 tiles one after the other, a tile's sums within 64 roundings
    tol = 2.0 ** -8 * (A + ref.abs()) + A * (2 * dz + 2200 * 2.0 ** -24 + 2.0 ** -20)
    assert bool(((out[0].cpu().double() - ref).abs() <= tol).all())
    rl = torch.logsumexp(z, -1) + math.log(n // 16)
    assert bool(((lse[0].cpu().double() - rl).abs() <= dz[:, 0] + 2200 * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * rl).all())
    c.keys[0] = None  # the others, as a short batch has them
    out[0], lse[0] = 0, -math.inf
    c.check(out, lse)


def test_graphs_streams_and_workspaces(skv):
    """Captured calls replay on new queries and lengths; two graphs share a workspace when replayed
    one after the other; two streams run at once with a workspace each."""
    c1 = Case(skv, 9, 2, 8, 900, _tails(9, 900, 200, 11), seed=11, cap=1100)
    c2 = Case(skv, 4, 4, 4, 350, _tails(4, 350, 100, 12), seed=12, cap=450)
    s1, s2 = skv.PrefixStep(c1.p, c1.pool, c1.prefix), skv.PrefixStep(c2.p, c2.pool, c2.prefix)
    ws = torch.empty(max(s1.ws.numel(), s2.ws.numel()), dtype=torch.uint8, device="cuda")
    q1, q2 = c1.qd.clone(), c2.qd.clone()
    outs = [(torch.empty_like(s.out), torch.empty_like(s.lse)) for s in (s1, s2)]
    graphs = []
    for c, q, o in ((c1, q1, outs[0]), (c2, q2, outs[1])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            skv.skv_prefix_attn(c.p, q, c.pool, c.prefix, o[0], o[1], ws)
        graphs.append(g)
    for it in range(3):
        for c, q in ((c1, q1), (c2, q2)):
            q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(it)).to(torch.bfloat16))
        c1.seq_lens[it] = 0
        c1.keys[it] = None
        for g in graphs + graphs[::-1]:
            g.replay()
        for c, q, o in ((c1, q1, outs[0]), (c2, q2, outs[1])):
            c.check(o[0], o[1], q=q.cpu())
    # two streams at once
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = [o[0].clone() for o in outs]
    torch.cuda.synchronize()
    for _ in range(20):
        s1.run(q1, stream=a)
        s2.run(q2, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(s1.out, want[0]) and torch.equal(s2.out, want[1])


def test_append_then_attend(skv):
    """A decode loop: every step's new token is normed, rotated and appended, then its query attends
    the shared prefix and the request's own tail (the prefix ends inside a block)."""
    B, H, G, P, steps = 6, 2, 4, 200, 20
    c = Case(skv, B, H, G, P, [P] * B, seed=13, cap=P + steps)
    g = torch.Generator().manual_seed(14)
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
    gq, gkk = ((1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2))
    rot = skv.Rotary(inv.cuda(), rot_dim=D, q_gamma=gq.cuda(), k_gamma=gkk.cuda())
    tok = skv.TokenStep(c.p, rot, c.pool)
    att = skv.PrefixStep(c.p, c.pool, c.prefix)

    def turned(x, gamma, pos):
        x = x.double()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma.double()
        ang = pos.double()[:, None, None] * inv.double()
        a, b = x[..., :64], x[..., 64:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    lens = [P] * B
    for it in range(steps):
        if it % 5 == 4:  # a finished request leaves its row of the batch unused
            lens[it // 5] = 0
            c.keys[it // 5] = None
        lens = [x + 1 if x else 0 for x in lens]
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q, k, v = (torch.randn((B, h, D), generator=g).to(torch.bfloat16) for h in (H * G, H, H))
        q_out = tok.append(q.cuda(), k.cuda(), v.cuda(), q_out=torch.zeros((B, H * G, D), dtype=torch.bfloat16,
                                                                           device="cuda"))
        out, lse = att.run(q_out)
        live = [b for b in range(B) if lens[b]]
        pos = torch.tensor([max(x - 1, 0) for x in lens])
        want_q, want_k = turned(q, gq, pos), turned(k, gkk, pos)
        for b in live:
            at = lens[b] - 1
            row = c.pool.gpu_k[int(c.pool.slot_table[b, at // 16]), :, at % 16].cpu()
            # half a step of bf16, and 48 roundings of 2^-24 of rows below 16 in size
            assert bool(((row.double() - want_k[b]).abs() <= 2.0 ** -8 * want_k[b].abs() + 2.0 ** -14).all())
            c.keys[b] = torch.cat([c.keys[b], row[None]])
            c.vals[b] = torch.cat([c.vals[b], v[b:b + 1]])
        err = (q_out.cpu().double() - want_q).abs()
        assert bool((err <= 2.0 ** -8 * want_q.abs() + 2.0 ** -14)[live].all())
        c.check(out, lse, q=q_out.cpu())
    assert int(tok.status.item()) == 0 and int(att.status.item()) == 0


def test_a_loop_of_calls_longer_than_the_ring_of_launches(skv):
    """Calls back to back on one stream, the workspace and the output shared: every launch waits for
    the one before, so the last call's result is the last input's."""
    c = Case(skv, 12, 2, 8, 700, _tails(12, 700, 200, 17), seed=17)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    qs = [torch.randn(c.q.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(5)]
    want = []
    for q in qs:
        out, lse = step.run(q)
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    for i in range(40):
        out, lse = step.run(qs[i % 5])
        got = out.clone(), lse.clone()
        assert torch.equal(got[0], want[i % 5][0]) and torch.equal(got[1], want[i % 5][1])
    for i in range(40):
        step.run(qs[i % 5])
    assert torch.equal(step.out, want[4][0]) and int(step.status.item()) == 0


def test_refuses_what_is_not_on_the_gpu(skv):
    c = Case(skv, 2, 1, 4, 40, [50, 60], seed=18)
    step = skv.PrefixStep(c.p, c.pool, c.prefix)
    n0 = skv.lib().skv_launch_count()
    with pytest.raises(ValueError):
        step.run(c.q)
    with pytest.raises(ValueError):
        skv.PrefixStep(c.p, c.pool, skv.Prefix(c.ptable, 40))
    with pytest.raises(ValueError):
        skv.skv_prefix_attn(c.p, c.qd, c.pool, c.prefix, step.out, step.lse.cpu(), step.ws)
    assert skv.lib().skv_launch_count() == n0
