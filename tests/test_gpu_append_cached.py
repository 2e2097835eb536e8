"""Appends beside a slot cache: a row that lands in a cached block (or token) is still there when the
block has been evicted and is read from the host pool again."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


B, CAP, NL = 2, 160, 16


class Side:
    """One copy of the history on the host, attended through `slots` GPU slots (0: none are used)."""

    def __init__(self, skv, latent, dtype, host, slots, lens):
        H, Hq, d, dv, bs = (1, 128, 576, 512, 1) if latent else (2, 8, 128, 128, 16)
        self.skv, self.latent, self.H, self.bs, self.d, self.dv = skv, latent, H, bs, d, dv
        per = CAP // bs
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.host = [None if t is None else t.clone().pin_memory() for t in host]
        rows = torch.arange(B * per, dtype=torch.int32).view(B, per)
        table = -rows - 1 if latent else (-rows - 1)[:, None].expand(B, H, per)
        shape = (slots, 1, 1, d) if latent else (slots, bs, d)
        gpu = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(1 if latent else 2)]
        self.pool = skv.Pool(gpu[0], None if latent else gpu[1], table.contiguous().cuda(), self.host[0], self.host[1],
                             table_heads=0 if latent else 1)
        self.p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=dv, max_len=CAP, topk=0, n_sink=0,
                             n_local=NL, block_size=bs, seq_lens=self.lens, d_idx=128, n_idx_q_heads=Hq,
                             dtype=skv.SKV_DTYPE_F32 if dtype == torch.float32 else skv.SKV_DTYPE_BF16)
        g = torch.Generator().manual_seed(9)
        self.q = torch.randn((B, Hq, d), generator=g).to(dtype).cuda()
        q_score, index = None, skv.IndexSrc()
        if latent:
            q_score = torch.randn((B, Hq, 128), generator=g).to(dtype).cuda()
            index = skv.IndexSrc(skv.SKV_INDEX_CONTIG, torch.zeros((B, 1, CAP, 128), dtype=dtype, device="cuda"))
        self.step = skv.DecodeStep(self.p, self.pool, self.q, index, q_score=q_score,
                                   out_dtype=dtype)
        self.tokens = skv.TokenStep(self.p, skv.Rotary(None), self.pool)

    def append(self, k, v, positions, requests):
        ids = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (positions, requests)]
        self.tokens.append(None, k, v, *ids)

    def entry(self, b, t):
        """The slot-table entries of position t, a head each."""
        tb = self.pool.slot_table.cpu().view(B, -1, CAP // self.bs)
        return tb[b, :, t // self.bs]

    def host_row(self, b, t):
        return [None if x is None else x[b * (CAP // self.bs) + t // self.bs, :, t % self.bs] for x in self.host]


def _host(latent, dtype):
    g = torch.Generator().manual_seed(3)
    H, d, dv, bs = (1, 576, 512, 1) if latent else (2, 128, 128, 16)
    n = B * CAP // bs
    k = torch.randn((n, H, bs, d), generator=g).to(dtype)
    return k, None if latent else torch.randn((n, H, bs, dv), generator=g).to(dtype)


def _token(side, seed, n, dtype):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((n, side.H, side.d), generator=g).to(dtype).cuda()
    return k, None if side.latent else torch.randn((n, side.H, side.dv), generator=g).to(dtype).cuda()


@pytest.mark.parametrize("latent,dtype", [(False, torch.bfloat16), (False, torch.float32), (True, torch.bfloat16)])
def test_promote_append_evict_read(skv, latent, dtype):
    lens = [70, 100]
    slots = 32 if latent else 8  # the two requests' local windows
    host = _host(latent, dtype)
    a = Side(skv, latent, dtype, host, slots, lens)
    ref = Side(skv, latent, dtype, host, 1, lens)  # every row in the host pool, no cache
    a.step.enable_cache(slots // 2)  # a step's promotions take the slots of the oldest use
    a.step.run_cached()
    a.step.run_cached()
    assert bool((a.entry(0, 69) >= 0).all()) and bool((a.entry(1, 99) >= 0).all())  # promoted
    # three tokens each, into blocks that have slots, and positions written a second time
    for i in range(3):
        for s in (a, ref):
            s.lens.add_(1)
            k, v = _token(s, 20 + i, 4, dtype)
            s.append(k, v, [70 + i, 100 + i, 60, 95 + i], [0, 1, 0, 1])
        a.step.run_cached()
        ref.step.run()
        assert torch.equal(a.step.out, ref.step.out) and torch.equal(a.step.lse, ref.step.lse)
    # request 0 pauses, request 1 attends elsewhere: every slot goes to other blocks
    for end in (40, 152):
        a.lens.copy_(torch.tensor([0, end], dtype=torch.int32))
        a.step.run_cached()
    assert bool((a.entry(0, 60) < 0).all()) and bool((a.entry(0, 72) < 0).all()) and bool((a.entry(1, 97) < 0).all())
    a.lens.copy_(ref.lens)
    a.step.run()
    ref.step.run()
    torch.cuda.synchronize()
    assert torch.equal(a.step.out, ref.step.out) and torch.equal(a.step.lse, ref.step.lse)
    for x, y in zip(a.host, ref.host):
        assert x is None or torch.equal(x, y)
    assert int(a.step.status.item()) == 0 and int(a.tokens.status.item()) == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("latent,dtype", [(False, torch.bfloat16), (False, torch.float32), (True, torch.bfloat16)])
def test_slot_and_host_row_are_written(skv, latent, dtype, graph):
    """Tokens of both tiers and padding: a row in a slot is the row behind it, what no token names stays."""
    slots = 64 if latent else 12
    a = Side(skv, latent, dtype, _host(latent, dtype), slots, [70, 100])
    a.step.enable_cache(slots)
    a.step.run_cached()  # the local windows have slots now
    torch.cuda.synchronize()
    before = [None if x is None else x.clone() for x in a.host]
    slot0 = a.pool.gpu_k.clone()
    pos, req = [69, 3, -1, 99, 98, 150, 64], [0, 0, 0, 1, 1, 1, -1]
    q = torch.randn((7, a.p.n_q_heads, a.d), generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    k, v = _token(a, 6, 7, dtype)
    ids = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (pos, req)]
    q_out = torch.full_like(q, 4.0)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.tokens.append(q, k, v, *ids, q_out=q_out)
        g.replay()
    else:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a.tokens.append(q, k, v, *ids, q_out=q_out, stream=side)
    torch.cuda.synchronize()
    want = before
    for i, (t, b) in enumerate(zip(pos, req)):
        live = t >= 0 and b >= 0
        assert torch.equal(q_out[i], q[i] if live else torch.full_like(q[i], 4.0))
        if not live:
            continue
        at = b * (CAP // a.bs) + t // a.bs
        want[0][at, :, t % a.bs] = k[i].cpu()
        if v is not None:
            want[1][at, :, t % a.bs] = v[i].cpu()
        entries = a.entry(b, t).tolist()
        assert all(e >= 0 for e in entries) == (i in (0, 3, 4))
        for h, e in enumerate(entries):
            if e >= 0:
                slot0[e].view(-1, a.d)[t % a.bs] = k[i, h]
    assert torch.equal(a.pool.gpu_k, slot0)
    for x, y in zip(a.host, want):
        assert x is None or torch.equal(x, y)
    assert int(a.tokens.status.item()) == 0


def test_the_plain_append_refuses_a_cached_pool(skv):
    a = Side(skv, False, torch.bfloat16, _host(False, torch.bfloat16), 4, [70, 100])
    k, v = _token(a, 1, 2, torch.bfloat16)
    skv.skv_append_kv(a.p, skv.Rotary(None), None, k, v, a.pool, None)
    a.step.enable_cache(4)
    n0 = skv.lib().skv_launch_count()
    with pytest.raises(ValueError):
        skv.skv_append_kv(a.p, skv.Rotary(None), None, k, v, a.pool, None)
    assert skv.lib().skv_launch_count() == n0
    skv.skv_append_kv_cached(a.p, skv.Rotary(None), None, k, v, a.pool, None)
    torch.cuda.synchronize()
    assert skv.lib().skv_launch_count() == n0 + 2
    for b, t in ((0, 69), (1, 99)):
        kr, vr = a.host_row(b, t)
        assert torch.equal(kr, k[b].cpu()) and torch.equal(vr, v[b].cpu())
