"""Block tables and slot maps from request lengths, against Python lists; and a run of them with
appends and decode steps over a cache in 4 bits."""

import numpy as np
import pytest
import torch

import kv4_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


class Model:
    """The rules of skv_update_tables, one request at a time."""

    def __init__(self, B, max_len, bs, n_blocks, stack, base=0, per=None):
        self.B, self.max_len, self.bs, self.n_blocks, self.base = B, max_len, bs, n_blocks, base
        self.table = np.full((B, per or -(-max_len // bs)), -7, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.stack = list(stack)
        self.status = 0

    def blocks(self, L):
        return range(self.base // self.bs, -(-L // self.bs)) if L > self.base else range(self.base // self.bs, self.base // self.bs)

    def update(self, n_new, n_tokens):
        pos, req = np.full(n_tokens, -1, np.int32), np.full(n_tokens, -1, np.int32)
        slots = np.full(n_tokens, -1, np.int64)
        lens, back, want = self.lens.copy(), [], []
        row = asked = 0
        for b in range(self.B):
            L, n = int(self.lens[b]), int(n_new[b])
            bad = L < 0 or L > self.max_len or 0 < L < self.base
            if n == 0:
                continue
            if n < 0:
                if bad:
                    self.status |= 4
                    continue
                left = max(L + n, 0)
                left = left if left > self.base else 0
                gone = [j for j in self.blocks(L) if j not in self.blocks(left)]
                back += [(b, j) for j in gone]
                lens[b] = left
                continue
            first, mine = row, n
            row += n
            if bad or (L or self.base) + n > self.max_len:
                self.status |= 4
                continue
            s = L or self.base
            fresh = [j for j in self.blocks(s + n) if j not in self.blocks(L)]
            asked += len(fresh)
            want.append((b, s, n, first, fresh, asked))
        for b, j in back:
            if not 0 <= self.table[b, j] < self.n_blocks:
                self.status |= 1
        stack = self.stack + [int(self.table[b, j]) for b, j in reversed(back)]
        free = len(stack)
        for b, s, n, first, fresh, asked in want:
            if first + n > n_tokens:
                self.status |= 2
            elif fresh and asked > free:
                self.status |= 16
            else:
                for j in fresh:
                    self.table[b, j] = stack.pop()
                lens[b] = s + n
                for i in range(n):
                    t = s + i
                    pos[first + i], req[first + i] = t, b
                    slots[first + i] = int(self.table[b, t // self.bs]) * self.bs + t % self.bs
        if len(stack) > self.n_blocks:
            self.status |= 1
            stack = stack[:self.n_blocks]
        self.stack, self.lens = stack, lens
        return pos, req, slots


class Pair:
    def __init__(self, skv, B, max_len, bs, n_blocks, base=0, seed=0, per=None, n_free=None):
        rng = np.random.default_rng(seed)
        self.skv, self.rng = skv, rng
        n_free = n_blocks if n_free is None else n_free
        stack = rng.permutation(n_blocks)[:n_free]
        self.m = Model(B, max_len, bs, n_blocks, stack.tolist(), base, per)
        free = torch.full((n_blocks,), -1, dtype=torch.int32)
        free[:n_free] = torch.from_numpy(stack.astype(np.int32))
        p = skv.Problem(batch=B, n_kv_heads=1, n_q_heads=1, d_qk=128, d_v=128, max_len=max_len, topk=0, n_sink=0,
                        n_local=0, block_size=bs, seq_lens=torch.zeros(B, dtype=torch.int32, device="cuda"))
        self.t = skv.BlockTables(p, torch.from_numpy(self.m.table).cuda(), free.cuda(), n_free=n_free, base=base)

    def update(self, n_new, n_tokens, stream=None):
        n_new = np.asarray(n_new, np.int32)
        got = self.t.update(torch.from_numpy(n_new).cuda(), n_tokens)
        want = self.m.update(n_new, n_tokens)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w)
        self.same()
        return got

    def same(self):
        m, t = self.m, self.t
        assert np.array_equal(t.tables.slot_table.cpu().numpy(), m.table)
        assert np.array_equal(t.p.seq_lens.cpu().numpy(), m.lens)
        assert t.state.tolist() == [len(m.stack), 0, 0, 0]
        assert t.tables.free_blocks[:len(m.stack)].tolist() == m.stack
        assert int(t.status.item()) == m.status


@pytest.mark.parametrize("B,max_len,bs,base,n_blocks", [
    (1, 1, 1, 0, 1), (1, 100, 16, 0, 7), (5, 200, 16, 0, 60), (5, 200, 16, 40, 60), (7, 90, 1, 13, 700),
    (64, 500, 32, 0, 900), (300, 300, 16, 100, 3000), (1500, 60, 16, 0, 4000), (4096, 40, 16, 17, 9000),
])
def test_random_steps(skv, B, max_len, bs, base, n_blocks):
    s = Pair(skv, B, max_len, bs, n_blocks, base, seed=B)
    rng = s.rng
    for i in range(12):
        kind = rng.random(B)
        room = np.maximum(max_len - np.where(s.m.lens > 0, s.m.lens, base), 0)
        n = np.where(kind < 0.5, np.minimum(rng.integers(0, max(2, max_len // 3), B), room),
                     np.where(kind < 0.8, 0, -rng.integers(0, max_len + 2, B)))
        if i % 4 == 3:
            n = np.where(kind < 0.1, room + 1, n)  # past max_len
        tokens = int(np.maximum(n, 0).sum())
        s.update(n, [tokens, tokens + 5, max(tokens - 3, 0), tokens][i % 4])


def test_no_blocks(skv):
    """Too few blocks: the requests that they suffice for, in order; those that need none get their tokens."""
    s = Pair(skv, 4, 100, 16, 8)
    s.update([16, 40, 60, 3], 119)   # 1 + 3 + 4 blocks and none left for the last
    assert int(s.t.status.item()) == skv.SKV_DEV_NO_BLOCK and s.m.lens.tolist() == [16, 40, 60, 0]
    s.update([1, 5, 4, 0], 10)       # the first needs one, the others none
    assert s.m.lens.tolist() == [16, 45, 64, 0]
    s.update([40, -45, 5, 30], 75)   # what one gives back serves the others in the same call: 3 blocks
    s.update([-100, -100, -100, -100], 0)
    assert sorted(s.m.stack) == list(range(8)) and s.m.lens.tolist() == [0, 0, 0, 0]


def test_taken_back(skv):
    """A call that takes back what the call before gave leaves lengths and stack as they were."""
    s = Pair(skv, 50, 400, 16, 1300, base=33, seed=4)
    s.update(s.rng.integers(0, 150, 50), 50 * 150)
    stack, lens = list(s.m.stack), s.m.lens.copy()
    n = s.rng.integers(0, 200, 50)
    s.update(n, 50 * 200)
    s.update(np.where(s.m.lens > lens, -n, 0), 0)
    assert s.m.stack == stack and np.array_equal(s.m.lens, lens)


def test_bad_state(skv):
    """Lengths that are none, entries that are no block, a stack with no room: flagged, and nothing out of place."""
    s = Pair(skv, 6, 100, 16, 40, base=20)
    s.update([30, 30, 30, 30, 30, 0], 150)
    for b, L in ((0, -5), (1, 101), (2, 10)):
        s.m.lens[b] = L
    s.t.p.seq_lens.copy_(torch.from_numpy(s.m.lens))
    s.update([1, 1, 1, 1, -1, 0], 4)
    s.update([-1, -1, -1, 0, 0, 0], 0)
    assert int(s.t.status.item()) == skv.SKV_DEV_BAD_LENGTH
    s.m.table[3, 1] = s.m.table[4, 2] = 40
    s.m.table[4, 1] = -2
    s.t.tables.slot_table.copy_(torch.from_numpy(s.m.table))
    s.update([0, 0, 0, -100, -100, 0], 0)
    assert int(s.t.status.item()) & skv.SKV_DEV_BAD_SLOT
    # more blocks come back than there are
    s = Pair(skv, 2, 64, 16, 6)
    s.update([64, 0], 64)
    s.m.stack = list(range(6))
    s.t.tables.free_blocks.copy_(torch.arange(6, dtype=torch.int32))
    s.t.state[0] = 6
    s.update([-64, 0], 0)
    assert int(s.t.status.item()) == skv.SKV_DEV_BAD_SLOT


def test_many_tokens(skv):
    s = Pair(skv, 3, 1 << 20, 16, 1 << 17)
    s.update([500001, 0, 777777], 1300000)
    s.update([-400000, 5, 100], 105)


def test_outputs_and_graph(skv):
    """Given outputs, no slots, two graphs over one state in turn, another stream."""
    s = Pair(skv, 8, 300, 16, 160)
    n_new = torch.tensor([1, 2, 0, 1, 3, 1, 1, 0], dtype=torch.int32, device="cuda")
    back = -n_new
    out = (torch.empty(12, dtype=torch.int32, device="cuda"), torch.empty(12, dtype=torch.int32, device="cuda"), None)
    s.t.update(n_new, 12, out=out)
    want = s.m.update(n_new.cpu().numpy(), 12)
    assert np.array_equal(out[0].cpu().numpy(), want[0]) and np.array_equal(out[1].cpu().numpy(), want[1])
    s.same()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        s.t.update(n_new, 12, out=out)
    with torch.cuda.graph(graphs[1]):
        s.t.update(back)
    for i in (0, 0, 1, 0, 0, 1, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        want = s.m.update((n_new, back)[i].cpu().numpy(), 12 if i == 0 else 0)
        if i == 0:
            assert np.array_equal(out[0].cpu().numpy(), want[0])
        s.same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rows = s.t.update(n_new, 9, stream=side)
    side.synchronize()
    assert np.array_equal(rows[2].cpu().numpy(), s.m.update(n_new.cpu().numpy(), 9)[2])
    s.same()


@pytest.mark.parametrize("group,bs", [(32, 16), (64, 32), (128, 64)])
def test_serving_run(skv, group, bs):
    """Prompts arrive, decode, one is taken back, one leaves and another comes: tables, appends and
    attention in 4 bits as a serving loop calls them, captured nowhere and checked every step."""
    B, H, G, D = 5, 2, 4, 128
    max_len, n_blocks = 400, 60 * 16 // bs
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=max_len, topk=24, n_sink=4,
                    n_local=16, block_size=bs, seq_lens=lens)
    table = torch.zeros((B, -(-max_len // bs)), dtype=torch.int32, device="cuda")
    pool = skv.Kv4Pool.empty(n_blocks, H, bs, table, group=group)
    pool.gpu_k.fill_(0xFF), pool.gpu_v.fill_(0xFF)
    tables = skv.BlockTables(p, table, torch.arange(n_blocks, dtype=torch.int32, device="cuda"))
    tokens, step = skv.TokenStep(p, skv.Rotary(None), pool), skv.Kv4Step(p, pool)
    g = torch.Generator().manual_seed(group)
    held = [[[[] for _ in range(H)] for _ in range(B)] for _ in range(2)]  # the rows each history should hold
    for news in ([100, 33, 0, 17, 64], [1, 1, 0, 1, 1], [3, 3, 50, 3, 3], [-2, 0, -1, -3, 0], [1, 0, 1, 1, 1],
                 [-400, 1, 1, 1, -400], [20, 1, 1, 1, 90], [1, 1, 1, 1, 1]):
        n = sum(max(x, 0) for x in news)
        at, req, _ = tables.update(torch.tensor(news, dtype=torch.int32, device="cuda"), n + 3)
        rows = torch.randn((n + 3, (H * G + 2 * H), D), generator=g).to(torch.bfloat16)
        dev = rows.cuda()
        tokens.append(dev[:, :H * G], dev[:, H * G:H * G + H], dev[:, H * G + H:], at, req)
        i = 0
        for b, x in enumerate(news):
            for kv in range(2):
                for h in range(H):
                    if x < 0:
                        del held[kv][b][h][x:]
                    else:
                        held[kv][b][h] += list(rows[i:i + x, H * G + kv * H + h].double().numpy())
            i += max(x, 0)
        cur = [len(held[0][b][0]) for b in range(B)]
        assert lens.tolist() == cur
        q = torch.randn((B, H * G, D), generator=g).to(torch.bfloat16)
        out, lse = (x.double().cpu().numpy() for x in step.attend_all(q.cuda()))
        sparse = step.run(q.cuda())[0].double().cpu().numpy()
        idx = step.idx.cpu().numpy()
        for b in range(B):
            for h in range(H):
                kv = [kv4_ref.quantise(np.array(held[i][b][h]).reshape(-1, D), group) if cur[b] else
                      tuple(np.zeros((0, w)) for w in (D, D // group, D // group)) for i in range(2)]
                hs = slice(h * G, (h + 1) * G)
                ref, rl, tol, tl = kv4_ref.attention(q[b, hs].double().numpy(), *kv, D ** -0.5)
                assert np.all(np.abs(out[b, hs] - ref) <= tol + 1e-37)
                if cur[b]:
                    assert np.all(np.abs(lse[b, hs] - rl) <= tl)
                sel = kv4_ref.attended(cur[b], 4, 16, [t for t in idx[b, h] if t >= 0])
                ref, _, tol, _ = kv4_ref.attention(q[b, hs].double().numpy(), *([a[sel] for a in side] for side in kv), D ** -0.5)
                assert np.all(np.abs(sparse[b, hs] - ref) <= tol + 1e-37)
    assert int(tables.status.item()) == int(tokens.status.item()) == int(step.status.item()) == 0
