"""Block tables in front of the 16-bit path -- update_tables, append, decode step and shared-prefix attention, nothing
waiting between -- and requests that hold a prefix alone."""

import numpy as np
import pytest
import torch

from test_gpu_tables import Pair

pytestmark = pytest.mark.gpu

D = 128
NEWS = [[5, 17, 0, 64, 1, 30], [1, 1, 0, 1, 1, 1], [1, -3, 50, 1, -400, 1], [1, 1, 1, -2, 0, 1],
        [-400, 1, 1, 1, 20, 1], [7, 1, 1, 1, 1, 1], [1, 16, 33, -400, 1, 1], [1, 1, 1, 90, 1, -20]]


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


@pytest.mark.parametrize("base", [0, 16, 55])
@pytest.mark.parametrize("bs", [16, 32])
def test_length_of_base(skv, base, bs):
    """A request that holds the prefix alone has no block of its own yet: it grows as one of length 0 does, and has
    nothing to give back."""
    s = Pair(skv, 5, 200, bs, 50, base=base)
    for lens in ([base] * 5, [base, 0, base, 0, base]):
        s.m.lens[:] = lens
        s.t.p.seq_lens.copy_(torch.from_numpy(s.m.lens))
        s.update([-1, -7, -200, 0, 0], 0)
        assert s.m.lens[:3].tolist() == [0, 0, 0] and len(s.m.stack) == 50
        s.m.lens[:] = lens
        s.t.p.seq_lens.copy_(torch.from_numpy(s.m.lens))
        s.update([1, 40, 0, 3, 64], 120)
        assert s.m.lens.tolist() == [base + 1, base + 40, lens[2], base + 3, base + 64]
        s.update([-200] * 5, 0)
        assert len(s.m.stack) == 50 and int(s.t.status.item()) == 0


class Serving:
    """A batch that shares `base` positions, blocks of 16 bits, and what each request should hold."""

    def __init__(self, skv, base, bs):
        self.skv, self.base, self.bs = skv, base, bs
        self.B, self.H, self.G, self.max_len = len(NEWS[0]), 2, 4, 256
        B, H, G = self.B, self.H, self.G
        g = torch.Generator().manual_seed(base + bs)
        shared = -(-base // bs)  # the prefix's blocks come first
        n = 8 + B * -(-self.max_len // bs)
        make = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
        self.k, self.v = make(n, H, bs, D).cuda(), make(n, H, bs, D).cuda()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        table = torch.full((B, -(-self.max_len // bs)), -1, dtype=torch.int32)
        table[:, :base // bs] = torch.arange(base // bs)
        self.table = table.cuda()
        self.p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=self.max_len,
                             topk=self.max_len, n_sink=4, n_local=16, block_size=bs, seq_lens=self.lens)
        pool = skv.Pool(self.k, self.v, self.table)
        free = torch.cat([torch.arange(shared, n), torch.zeros(shared, dtype=torch.int64)]).int().cuda()
        self.tables = skv.BlockTables(self.p, self.table, free, n_free=n - shared, base=base)
        self.tokens = skv.TokenStep(self.p, skv.Rotary(None, rot_dim=0), pool)
        self.decode = skv.DecodeStep(self.p, pool, torch.zeros((B, H * G, D), dtype=torch.bfloat16, device="cuda"),
                                     skv.IndexSrc(skv.SKV_INDEX_PAGED))
        prefix = torch.arange(shared, dtype=torch.int32, device="cuda") if base else None
        self.prefix = skv.PrefixStep(self.p, pool, skv.Prefix(prefix, base))
        self.n_new = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in NEWS]
        self.count = [sum(max(y, 0) for y in x) + 2 for x in NEWS]
        self.rows = [make(n, 2 * H, D).cuda() for n in self.count]
        self.q = [make(B, H * G, D).cuda() for _ in NEWS]
        # what a request holds after each step, and the requests that come with it
        self.held, self.come = [], []
        cur = [[torch.zeros((0, 2 * H, D), dtype=torch.float64)] for _ in range(B)]
        for news, rows in zip(NEWS, self.rows):
            i, rows = 0, rows.double().cpu()
            self.come.append(torch.tensor([b for b, x in enumerate(news) if x > 0 and len(torch.cat(cur[b])) == 0],
                                          dtype=torch.int64, device="cuda"))
            for b, x in enumerate(news):
                if x < 0:
                    cur[b] = [torch.cat(cur[b])[:x]]
                cur[b].append(rows[i:i + max(x, 0)])
                i += max(x, 0)
            self.held.append([torch.cat(x) for x in cur])

    def run(self, waits):
        wait = torch.cuda.synchronize if waits else lambda: None
        j, rest = self.base // self.bs, self.base % self.bs
        got = []
        for i, (n_new, n, rows, q, come) in enumerate(zip(self.n_new, self.count, self.rows, self.q, self.come)):
            at, req, _ = self.tables.update(n_new, n)
            wait()
            if rest and len(come):  # the rows of a block that the prefix ends inside, copied to each request's own
                own = self.table[come, j].long()
                for x in (self.k, self.v):
                    x[own, :, :rest] = x[j, :, :rest]
                wait()
            self.tokens.append(None, rows[:, :self.H], rows[:, self.H:], at, req)
            wait()
            self.decode.q.copy_(q)
            self.decode.run()
            wait()
            out, lse = self.prefix.run(q)
            wait()
            got.append([x.clone() for x in (self.decode.out, self.decode.lse, out, lse, self.lens, self.table)])
            wait()
        return got


@pytest.mark.parametrize("base,bs", [(0, 16), (48, 16), (40, 16), (71, 16)])
def test_tables_append_decode_prefix(skv, base, bs):
    """The decode step's selection takes every candidate, so it and the shared-prefix attention attend the same rows.

    Against 64 bits: weights are bf16 at V (2^-8 of the weighted |V|), outputs round once more; a logit has 160
    additions of 2^-23 of its parts, the sums n + 64 of theirs."""
    waited, s = Serving(skv, base, bs).run(True), Serving(skv, base, bs)
    got = s.run(False)
    torch.cuda.synchronize()
    for w, g in zip(waited, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
    H, G = s.H, s.G
    shared = [x[:-(-base // bs)].double().cpu().transpose(1, 2).reshape(-1, H, D)[:base] for x in (s.k, s.v)]
    for held, q, results in zip(s.held, s.q, got):
        d_out, d_lse, p_out, p_lse, lens, _ = (x.cpu() for x in results)
        q = q.double().cpu()
        for b in range(s.B):
            n = len(held[b])
            assert int(lens[b]) == (n + base if n else 0)
            if n == 0:
                for out, lse in ((d_out, d_lse), (p_out, p_lse)):
                    assert torch.all(out[b] == 0) and torch.all(torch.isneginf(lse[b]))
                continue
            for h in range(H):
                k, v = torch.cat([shared[0][:, h], held[b][:, h]]), torch.cat([shared[1][:, h], held[b][:, H + h]])
                x = q[b, h * G:(h + 1) * G]
                z, dz = x @ k.T * D ** -0.5, x.abs() @ k.abs().T * (D ** -0.5 * 160 * 2.0 ** -23)
                w = z.softmax(-1)
                ref, lref = w @ v, z.logsumexp(-1)
                rel = 2 * dz.amax(-1, keepdim=True) + 2.0 ** -20 + (n + base + 64) * 2.0 ** -23
                tol = (2.0 ** -8 + rel) * (w @ v.abs()) + 2.0 ** -8 * ref.abs()
                for out, lse in ((d_out, d_lse), (p_out, p_lse)):
                    assert torch.all((out[b, h * G:(h + 1) * G].double() - ref).abs() <= tol), (b, h)
                    assert torch.all((lse[b, h * G:(h + 1) * G].double() - lref).abs()
                                     <= rel[:, 0] + 2.0 ** -22 * lref.abs()), (b, h)
    for x in (s.tables, s.tokens, s.decode, s.prefix):
        assert int(x.status.item()) == 0
