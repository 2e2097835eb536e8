"""The cache in 4 bits on the GPU: append, gather, scores and attention against fp64 numpy.

Tolerances stand at kv4_ref.attention and at assert_scores / assert_coded below; those of the
rows before they are coded are test_gpu_tokens.reference's."""

import numpy as np
import pytest
import torch

import kv4_ref
from test_gpu_tokens import reference as token_reference

pytestmark = pytest.mark.gpu

D = 128
HALF = 2.0 ** -8  # of a bf16 rounding


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A batch with its histories in 4 bits; rows nobody wrote are NaN."""

    def __init__(self, skv, lens, H, G, group=32, bs=16, seed=0, host=0.0, per_head=False, scale=1.0, k=0, ns=0, nl=0,
                 agg=0, sm_scale=0.0, max_len=None, q_scale=1.0):
        self.skv, self.lens, self.H, self.G, self.group, self.bs = skv, lens, H, G, group, bs
        rng = np.random.default_rng(seed)
        self.rng = rng
        B = len(lens)
        self.max_len = max_len or max(max(lens), 1)
        per = -(-self.max_len // bs) + 1
        units = B * H if per_head else B
        n = units * per
        perm = rng.permutation(n).reshape(units, per)
        on_host = rng.random((units, per)) < host
        self.table = np.where(on_host, -perm - 1, perm).astype(np.int32)
        self.per_head = per_head
        # a GPU block of a per-head table holds one head; a host block every head
        self.gpu = [kv4_ref.Cache(n, 1 if per_head else H, bs, group, rng) for _ in range(2)]
        self.host = [kv4_ref.Cache(n, H, bs, group, rng) if host else None for _ in range(2)]
        self.rows = {}
        for b in range(B):
            for h in range(H):
                t = np.arange(lens[b])
                for kv in range(2):
                    x = scale * rng.standard_normal((lens[b], D)) * (0.25 + rng.random((lens[b], 1))) + 0.3 * rng.standard_normal(D)
                    self.write(kv, b, h, t, x)
                    self.rows[kv, b, h] = self.read(kv, b, h, t)
        self.q = torch.from_numpy(q_scale * rng.standard_normal((B, H * G, D))).to(torch.bfloat16)
        self.p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=self.max_len, topk=k,
                             n_sink=ns, n_local=nl, block_size=bs, seq_lens=_dev(np.array(lens, np.int32)),
                             group_agg=agg, sm_scale=sm_scale)
        self.scale = sm_scale or D ** -0.5
        self.upload()

    def place(self, b, h, t):
        e = self.table[b * self.H + h if self.per_head else b][t // self.bs]
        return e >= 0, np.where(e >= 0, e, -e - 1)

    def write(self, kv, b, h, t, x):
        gpu, e = self.place(b, h, t)
        if gpu.any():
            self.gpu[kv].put(e[gpu], 0 if self.per_head else h, t[gpu], x[gpu])
        if (~gpu).any():
            self.host[kv].put(e[~gpu], h, t[~gpu], x[~gpu])

    def read(self, kv, b, h, t, gpu_pool=None, host_pool=None):
        gpu, e = self.place(b, h, t)
        out = [np.zeros((len(t), w)) for w in (D, D // self.group, D // self.group)]
        for on, cache, head, pool in ((gpu, self.gpu[kv], 0 if self.per_head else h, gpu_pool),
                                      (~gpu, self.host[kv], h, host_pool)):
            if on.any():
                for o, v in zip(out, cache.raw(e[on], head, t[on], pool)):
                    o[on] = v
        return out

    def upload(self):
        gpu = [_dev(c.pool[:, 0] if self.per_head else c.pool) for c in self.gpu]
        host = [None if c is None else torch.from_numpy(c.pool).pin_memory() for c in self.host]
        table = self.table.reshape(len(self.lens), self.H, -1) if self.per_head else self.table
        self.pool = self.skv.Kv4Pool(gpu[0], gpu[1], _dev(table), host[0], host[1], table_heads=int(self.per_head),
                                     group=self.group)
        self.step = self.skv.Kv4Step(self.p, self.pool)

    def downloaded(self, kv):
        """Both tiers of K or V as numpy, in the references' shapes."""
        gpu = (self.pool.gpu_v if kv else self.pool.gpu_k).cpu().numpy()
        host = self.pool.host_v if kv else self.pool.host_k
        return gpu[:, None] if self.per_head else gpu, None if host is None else host.numpy()

    def unit(self, kv, b, h, at):
        at = np.asarray(at, dtype=np.int64)
        return [a[at] for a in self.rows[kv, b, h]]

    def check(self, out, lse, lists=None, units=None):
        """out and lse against fp64; lists(b, row): attended positions of a row (default: all)."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        per_q = self.p.group_agg == self.skv.SKV_AGG_HEAD and lists is not None
        for b in range(len(self.lens)):
            for row in range(self.H * self.G if per_q else self.H):
                if units is not None and (b, row) not in units:
                    continue
                h = row // self.G if per_q else row
                heads = [row] if per_q else list(range(h * self.G, (h + 1) * self.G))
                at = range(self.lens[b]) if lists is None else lists(b, row)
                ref, rl, tol, tl = kv4_ref.attention(self.q[b, heads].double().numpy(), self.unit(0, b, h, at),
                                                     self.unit(1, b, h, at), self.scale)
                err = np.abs(out[b, heads] - ref)
                assert np.all(err <= tol + 1e-37), (b, row, float((err - tol).max()), float(err.max()))
                if len(at) == 0:
                    assert np.all(np.isneginf(lse[b, heads])) and np.all(out[b, heads] == 0)
                else:
                    assert np.all(np.abs(lse[b, heads] - rl) <= tl), (b, row, np.abs(lse[b, heads] - rl).max(), tl)


@pytest.mark.parametrize("lens,H,G,kw", [
    ([1], 1, 1, {}),
    ([0, 1, 15, 16, 17, 0, 33], 2, 4, {}),
    ([300, 0, 77, 128], 3, 8, dict(group=64)),
    ([300, 5, 77, 129], 2, 16, dict(group=128, bs=48)),
    ([257, 4, 0, 1000], 2, 9, dict(bs=64)),
    ([600, 31], 2, 7, dict(group=64, bs=32, host=0.4)),
    ([600, 31, 100], 3, 5, dict(per_head=True, host=0.3)),
    ([90, 500], 2, 2, dict(per_head=True, bs=32, group=128)),
    ([5000, 1, 2500], 4, 8, {}),
    ([5000, 1, 2500], 2, 3, dict(group=128)),
    ([40000], 1, 8, dict(scale=0.01)),
    ([700, 700], 2, 4, dict(scale=1e6, q_scale=1e-5)),
    ([700, 90], 2, 4, dict(scale=1e-6, q_scale=1e5)),
    ([400, 90], 2, 12, dict(sm_scale=0.31)),
    ([7] * 300, 2, 4, {}),
])
def test_attend_all(skv, lens, H, G, kw):
    c = Case(skv, lens, H, G, **kw)
    out, lse = c.step.attend_all(c.q.cuda())
    c.check(out, lse)
    first = (out.clone(), lse.clone())
    again = c.step.attend_all(c.q.cuda())
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])  # the same bits
    assert int(c.step.status.item()) == 0


def _selection(c, rng, k, heads, holes=False):
    """Ascending candidate positions per row, -1 past their end (and in between where there are holes)."""
    idx = np.full((len(c.lens), heads, k), -1, np.int32)
    for b, L in enumerate(c.lens):
        lo = min(L, c.p.n_sink)
        hi = max(lo, L - c.p.n_local)
        for r in range(heads):
            n = min(k, hi - lo)
            sel = np.sort(rng.choice(hi - lo, n, replace=False) + lo) if n else np.zeros(0, np.int64)
            if holes:
                sel = np.where(rng.random(n) < 0.4, -1, sel)
            idx[b, r, :n] = sel
    return idx


@pytest.mark.parametrize("lens,H,G,k,ns,nl,kw", [
    ([1], 1, 1, 1, 0, 0, {}),
    ([0, 3, 70, 500], 2, 4, 50, 4, 64, {}),
    ([0, 3, 70, 500], 2, 8, 50, 0, 0, dict(group=64, bs=32)),
    ([900, 18, 200], 3, 16, 100, 16, 33, dict(group=128)),
    ([900, 18, 200], 2, 5, 100, 1, 7, dict(host=0.5, bs=48)),
    ([900, 18, 200], 2, 5, 100, 1, 7, dict(host=0.5, per_head=True)),
    ([900, 18, 200], 2, 5, 0, 20, 70, {}),
    ([3000, 2999], 4, 8, 700, 4, 128, {}),
    ([900, 18, 200], 2, 7, 90, 4, 30, dict(agg=2)),
    ([500, 44], 2, 7, 90, 4, 30, dict(agg=2, per_head=True, group=64)),
])
@pytest.mark.parametrize("holes", [False, True])
def test_attend_list(skv, lens, H, G, k, ns, nl, kw, holes):
    c = Case(skv, lens, H, G, k=k, ns=ns, nl=nl, **kw)
    heads = H * G if kw.get("agg") == 2 else H
    idx = _selection(c, np.random.default_rng(5), k, heads, holes)
    out, lse = c.step.attend(c.q.cuda(), _dev(idx))
    lists = lambda b, r: kv4_ref.attended(lens[b], ns, nl, [t for t in idx[b, r] if t >= 0])  # noqa: E731
    c.check(out, lse, lists)
    assert int(c.step.status.item()) == 0
    # the rows of the list, holes and ends zero
    kk, vv = c.step.gather(_dev(idx))
    n_att = ns + k + nl
    for b in range(len(lens)):
        for r in range(heads):
            full = kv4_ref.attended(lens[b], ns, nl, idx[b, r])
            full = np.array(full + [-1] * (n_att - len(full)), np.int64)
            for kv, got in ((0, kk), (1, vv)):
                want = kv4_ref.values(*c.unit(kv, b, r // G if heads != H else r, np.maximum(full, 0))) if lens[b] else np.zeros((n_att, D))
                want = want * (full >= 0)[:, None]
                err = np.abs(got[b, r].double().cpu().numpy() - want)
                assert np.all(err <= (HALF + 2.0 ** -23) * np.abs(want) + 1e-37)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gather_f32_window(skv, group):
    c = Case(skv, [100, 3, 0, 41], 2, 4, group=group, host=0.3)
    p = skv.Problem(**{**vars(c.p), "n_local": 37, "dtype": skv.SKV_DTYPE_F32})
    kk, vv = skv.Kv4Step(p, c.pool).gather()
    assert kk.shape == (4, 2, 37, D) and kk.dtype == torch.float32
    for b, L in enumerate(c.lens):
        at = np.arange(max(0, L - 37), L)
        for h in range(2):
            for kv, got in ((0, kk), (1, vv)):
                want = kv4_ref.values(*c.unit(kv, b, h, at))
                g = got[b, h].double().cpu().numpy()
                assert np.all(np.abs(g[:len(at)] - want) <= 2.0 ** -23 * np.abs(want) + 1e-37)
                assert np.all(g[len(at):] == 0)
    only = torch.empty_like(kk)
    skv.skv_gather_kv4(p, c.pool, None, None, only)
    assert torch.equal(only, vv)


def assert_scores(c, scores, q, agg, Gi, before):
    """160 additions of 2^-23 of sum |q| (15 s + 8 s + |z|), a mean's own 2 G more; the rest as it was."""
    got = scores.double().cpu().numpy()
    for b, L in enumerate(c.lens):
        lo = min(L, c.p.n_sink)
        hi = max(lo, L - c.p.n_local)
        for h in range(c.H):
            qh = q[b, h * Gi:(h + 1) * Gi].double().numpy()
            k, s, z = c.unit(0, b, h, np.arange(lo, hi))
            rep = lambda a: np.repeat(np.abs(a), c.group, -1)  # noqa: E731
            x, m = qh @ kv4_ref.values(k, s, z).T, np.abs(qh) @ (23 * rep(s) + rep(z)).T
            if agg == 0:
                x, m = x.mean(0, keepdims=True), m.mean(0, keepdims=True)
            elif agg == 1:
                x, m = x.max(0, keepdims=True), m.max(0, keepdims=True)
            rows = slice(h * Gi, (h + 1) * Gi) if agg == 2 else slice(h, h + 1)
            err = np.abs(got[b, rows, lo:hi] - x)
            assert np.all(err <= (160 + 2 * Gi) * 2.0 ** -23 * m), float((err / m).max() * 2 ** 23)
            assert np.all(got[b, rows, :lo] == before) and np.all(got[b, rows, hi:] == before)


@pytest.mark.parametrize("agg", [0, 1, 2])
@pytest.mark.parametrize("lens,H,G,ns,nl,kw", [
    ([1], 1, 1, 0, 0, {}),
    ([0, 3, 70, 500, 16, 17], 2, 4, 4, 13, {}),
    ([1000, 18, 200], 3, 16, 16, 33, dict(group=128, bs=32)),
    ([1000, 18, 200], 2, 9, 5, 0, dict(group=64, host=0.5)),
    ([300, 18], 2, 8, 0, 100, dict(per_head=True, bs=48)),
    ([6000, 5999], 2, 3, 4, 128, dict(scale=100.0)),
])
def test_score(skv, agg, lens, H, G, ns, nl, kw):
    c = Case(skv, lens, H, G, ns=ns, nl=nl, agg=agg, **kw)
    scores = torch.full((len(lens), H * G if agg == 2 else H, c.max_len), 7.0, device="cuda")
    assert c.step.score(c.q.cuda(), scores) is scores
    assert_scores(c, scores, c.q, agg, G, 7.0)
    assert int(c.step.status.item()) == 0


def test_score_other_heads(skv):
    """A scoring query with its own count of heads, more than a tile's columns."""
    c = Case(skv, [100, 37], 2, 4)
    q = torch.randn((2, 2 * 40, D)).to(torch.bfloat16)
    p = skv.Problem(**{**vars(c.p), "n_idx_q_heads": 80})
    scores = torch.zeros((2, 2, c.max_len), device="cuda")
    skv.skv_score_kv4(p, q.cuda(), c.pool, scores)
    assert_scores(c, scores, q, 0, 40, 0.0)


@pytest.mark.parametrize("agg,G,kw", [(0, 8, {}), (1, 8, dict(bs=32)), (2, 4, dict(group=64)), (0, 3, dict(per_head=True))])
def test_step(skv, agg, G, kw):
    """score, top-k and attention in one call are those calls in turn; the selection is exact on the scores."""
    c = Case(skv, [700, 90, 0, 300], 2, G, k=60, ns=4, nl=32, agg=agg, **kw)
    q = c.q.cuda()
    out, lse = c.step.run(q)
    heads = 2 * G if agg == 2 else 2
    scores, idx = c.step.scores.cpu().numpy(), c.step.idx.cpu().numpy()
    for b, L in enumerate(c.lens):
        lo = min(L, 4)
        hi = max(lo, L - 32)
        for r in range(heads):
            x = scores[b, r, lo:hi]
            want = np.sort(np.argsort(-x, kind="stable")[:60] + lo)
            assert np.array_equal(idx[b, r, :len(want)], want) and np.all(idx[b, r, len(want):] == -1)
    c.check(out, lse, lambda b, r: kv4_ref.attended(c.lens[b], 4, 32, [t for t in idx[b, r] if t >= 0]))
    one = skv.Kv4Step(c.p, c.pool)
    one.score(q)
    one.topk()
    a, l = one.attend(q)
    assert torch.equal(one.idx, c.step.idx) and torch.equal(a, out) and torch.equal(l, lse)
    c.check(*c.step.attend_all(q))  # whatever the selection
    assert int(c.step.status.item()) == 0 and int(one.status.item()) == 0


def test_bad_entries(skv):
    """Entries outside their pools: flagged, no weight, NaN scores, zero rows; positions outside the candidates too."""
    c = Case(skv, [200, 100], 2, 4, k=3, ns=4, nl=16)
    table = c.pool.slot_table.clone()
    n = c.pool.gpu_k.shape[0]
    table[0, 2], table[0, 5], table[1, 0] = n, -1, 2 ** 31 - 1  # past the pool; on a host that is not there
    c.pool.slot_table.copy_(table)
    out, lse = c.step.attend_all(c.q.cuda())
    gone = {0: set(range(32, 48)) | set(range(80, 96)), 1: set(range(16))}
    c.check(out, lse, lambda b, h: [t for t in range(c.lens[b]) if t not in gone[b]])
    assert int(c.step.status.item()) == skv.SKV_DEV_BAD_SLOT
    scores = c.step.score(c.q.cuda()).cpu().numpy()
    for b in range(2):
        for t in range(4, c.lens[b] - 16):
            assert np.all(np.isnan(scores[b, :, t])) == (t in gone[b])
    c.step.status.zero_()
    idx = np.full((2, 2, 3), 60, np.int32)
    idx[0, 0] = [3, 60, 61]      # the sink
    idx[0, 1] = [60, 61, 184]    # the window
    idx[1, :] = [50, 51, 2 ** 31 - 1]
    out, lse = c.step.attend(c.q.cuda(), _dev(idx))
    good = {(0, 0): [60, 61], (0, 1): [60, 61], (1, 0): [50, 51], (1, 1): [50, 51]}
    c.check(out, lse, lambda b, h: [t for t in kv4_ref.attended(c.lens[b], 4, 16, good[b, h]) if t not in gone[b]])
    assert int(c.step.status.item()) == skv.SKV_DEV_BAD_SLOT | skv.SKV_DEV_BAD_INDEX
    k, v = c.step.gather(_dev(idx))
    assert torch.all(k[0, 0, 4] == 0) and torch.all(v[0, 1, 6] == 0) and torch.all(k[1, :, :4] == 0)
    # every entry bad: an empty list
    c.pool.slot_table.fill_(n)
    out, lse = c.step.attend_all(c.q.cuda())
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_bad_lengths(skv):
    c = Case(skv, [50, 64, 20], 2, 4)
    c.p.seq_lens.copy_(torch.tensor([-3, 70, 20], dtype=torch.int32))
    out, lse = c.step.attend_all(c.q.cuda())
    assert int(c.step.status.item()) == skv.SKV_DEV_BAD_LENGTH
    c.lens = [0, 64, 20]  # below 0 counts as 0, past max_len as max_len
    c.check(out, lse)


def test_rows_that_are_not_numbers(skv):
    """A NaN in an attended value group reaches that group of the output alone, one in a key all of it;
    rows past the history (NaN in every case here) reach nothing."""
    c = Case(skv, [40, 40], 1, 4)
    gpu, e = c.place(0, 0, np.array([7]))
    cells, rows = c.gpu[1].cells(e, 0, np.array([7]))
    pool = c.pool.gpu_v.view(-1, c.gpu[1].cell)
    pool[int(cells[0]), 1024 + 4 * (int(rows[0]) * 4 + 2):1024 + 4 * (int(rows[0]) * 4 + 3)] = 0xFF
    out, lse = c.step.attend_all(c.q.cuda())
    assert torch.all(torch.isnan(out[0, :, 64:96])) and not torch.any(torch.isnan(out[0, :, :64])) \
        and not torch.any(torch.isnan(out[0, :, 96:])) and torch.all(torch.isfinite(lse))
    c.check(out, lse, units=[(1, 0)])
    gpu, e = c.place(0, 0, np.array([9]))
    cells, rows = c.gpu[0].cells(e, 0, np.array([9]))
    c.pool.gpu_k.view(-1, c.gpu[0].cell)[int(cells[0]), 1024 + 16 * int(rows[0]):1040 + 16 * int(rows[0])] = 0xFF
    out, lse = c.step.attend_all(c.q.cuda())
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
    c.check(out, lse, units=[(1, 0)])


@pytest.mark.parametrize("kind", ["constant", "zero", "rising", "falling", "spread"])
def test_hard_values(skv, kind):
    """Steps of 0, steps and maxima that rise (or fall) by orders of magnitude along the history."""
    c = Case(skv, [900], 2, 8, group=64)
    rng = np.random.default_rng(3)
    t = np.arange(900)
    for h in range(2):
        for kv in range(2):
            x = rng.standard_normal((900, D))
            if kind == "constant":
                x = np.full((900, D), 1.5) if kv else x
            elif kind == "zero":
                x = 0 * x
            elif kind in ("rising", "falling"):
                f = np.exp2((t if kind == "rising" else 899 - t) / 45.0)[:, None]
                x = x * (f if kv else f ** 0.2)
            else:
                x = x * np.exp2(rng.integers(-20, 20, (900, 1)) * (1.0 if kv else 0.1))
            c.write(kv, 0, h, t, x)
            c.rows[kv, 0, h] = c.read(kv, 0, h, t)
    c.upload()
    out, lse = c.step.attend_all(c.q.cuda())
    c.check(out, lse)


def test_small_scale(skv):
    """Zero queries under a scale that takes their logits' unit out of fp32: equal weights, masked rows none."""
    c = Case(skv, [23, 300], 2, 4, k=5, ns=4, nl=9, sm_scale=1e-30)
    c.q[:, ::3] = 0
    c.check(*c.step.attend_all(c.q.cuda()))
    idx = torch.tensor([[4, 9, 13, -1, -1], [5, 100, 17, 250, -1]], dtype=torch.int32).unsqueeze(1).repeat(1, 2, 1)
    c.check(*c.step.attend(c.q.cuda(), idx.contiguous().cuda()),
            lambda b, r: kv4_ref.attended(c.lens[b], 4, 9, [t for t in idx[b, r].tolist() if t >= 0]))
    assert int(c.step.status.item()) == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_query_that_is_no_number(skv, bad):
    """A query head with such an entry: NaN, and the other heads as without it."""
    c = Case(skv, [77, 1000], 2, 4, agg=2)
    want, lse = (x.clone() for x in c.step.attend_all(c.q.cuda()))
    c.q[0, 1, 40] = bad
    c.q[1, 6, 127] = bad
    out, l = c.step.attend_all(c.q.cuda())
    hit = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 6] = True
    assert out[hit].isnan().all() and l[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(l[~hit], lse[~hit])
    for agg in (0, 1, 2):
        p = skv.Problem(**{**vars(c.p), "group_agg": agg})
        scores = torch.zeros((2, 8 if agg == 2 else 2, c.max_len), device="cuda")
        skv.skv_score_kv4(p, c.q.cuda(), c.pool, scores)
        rows = hit if agg == 2 else hit.view(2, 2, 4).any(-1)
        for b, L in enumerate(c.lens):
            assert scores[b, rows[b], :L].isnan().all() and scores[b, ~rows[b], :L].isfinite().all()


def test_far_blocks(skv):
    """Blocks past 4 GB of the pool."""
    H, bs = 8, 16
    cell = skv.Kv4Pool.cell_bytes(32)
    n = 5 * 2 ** 30 // (H * cell)
    c = Case(skv, [100], H, 4)
    table = torch.tensor([[n - 1 - i for i in range(8)]], dtype=torch.int32, device="cuda")
    big = [torch.empty((n, H, 1, cell), dtype=torch.uint8, device="cuda") for _ in range(2)]
    src = torch.from_numpy(c.table[0, :8].astype(np.int64)).cuda()
    for a, b in zip(big, (c.pool.gpu_k, c.pool.gpu_v)):
        a[table[0].long()] = b[src]
    step = skv.Kv4Step(c.p, skv.Kv4Pool(*big, table))
    c.check(*step.attend_all(c.q.cuda()))
    del big, step


def test_streams_and_graphs(skv):
    c = Case(skv, [700, 90, 0, 300], 2, 4, k=60, ns=4, nl=32)
    q = c.q.cuda()
    want = [x.clone() for x in c.step.attend_all(q)]
    want_step = [x.clone() for x in c.step.run(q)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = skv.Kv4Step(c.p, c.pool)
    got = other.attend_all(q, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # captured twice over the same workspace, replayed in turn
    graphs = []
    for call in (lambda: c.step.attend_all(q), lambda: c.step.run(q)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _ in range(3):
        for g, w in zip(graphs, (want, want_step)):
            c.step.out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.step.out, w[0]) and torch.equal(c.step.lse, w[1])
    # lengths that change between replays
    c.p.seq_lens.copy_(torch.tensor([30, 0, 0, 299], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    c.lens = [30, 0, 0, 299]
    c.check(c.step.out, c.step.lse)


@pytest.mark.parametrize("seed", range(16))
def test_shapes_at_random(skv, seed):
    """Whole histories, lists, gathers and scores of batches, heads, groups, blocks and tables drawn together."""
    rng = np.random.default_rng(100 + seed)
    B = int(rng.choice([1, 2, 5, 17, 130, 400]))
    longest = int(rng.choice([1, 15, 16, 40, 600]) if B > 5 else rng.choice([1, 17, 300, 4000]))
    lens = [int(x) for x in rng.integers(0, longest + 1, B)]
    if rng.random() < 0.3:
        lens = [x if rng.random() < 0.2 else 0 for x in lens]
    H, G, agg = int(rng.integers(1, 4)), int(rng.integers(1, 17)), int(rng.integers(0, 3))
    per_head = bool(rng.random() < 0.4)
    k, ns, nl = int(rng.choice([0, 1, 16, 33, 200])), int(rng.choice([0, 1, 4, 19])), int(rng.choice([0, 1, 17, 128]))
    c = Case(skv, lens, H, G, k=k, ns=ns, nl=nl, agg=agg, group=int(rng.choice([32, 64, 128])),
             bs=int(rng.choice([16, 32, 48, 80, 256])), host=float(rng.choice([0.0, 0.0, 0.5])), per_head=per_head,
             max_len=longest + int(rng.integers(0, 100)), seed=seed)
    q = c.q.cuda()
    c.check(*c.step.attend_all(q))
    heads = H * G if agg == 2 else H
    idx = _selection(c, rng, k, heads, bool(rng.random() < 0.5))
    if k + ns + nl:
        out = [x.clone() for x in c.step.attend(q, _dev(idx))]
        c.check(*out, lambda b, r: kv4_ref.attended(lens[b], ns, nl, [t for t in idx[b, r] if t >= 0]))
        again = c.step.attend(q, _dev(idx))
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
        kk, vv = c.step.gather(_dev(idx))
        for b in {0, B // 2, B - 1}:
            if lens[b] == 0:
                assert not kk[b].any() and not vv[b].any()
                continue
            for r in range(heads):
                full = kv4_ref.attended(lens[b], ns, nl, idx[b, r])
                at = np.array(full + [-1] * (ns + k + nl - len(full)), np.int64)
                for kv, got in ((0, kk), (1, vv)):
                    want = kv4_ref.values(*c.unit(kv, b, r // G if agg == 2 else r, np.maximum(at, 0))) * (at >= 0)[:, None]
                    err = np.abs(got[b, r].double().cpu().numpy() - want)
                    assert np.all(err <= (HALF + 2.0 ** -23) * np.abs(want) + 1e-37)
    scores = torch.full((B, heads, c.max_len), 7.0, device="cuda")
    c.step.score(q, scores)
    assert_scores(c, scores, c.q, agg, G, 7.0)
    assert int(c.step.status.item()) == 0


def test_two_at_once(skv):
    """Steps of their own over one pool, on two streams, none waiting for the other."""
    c = Case(skv, [3000, 90, 0, 2000], 2, 8, k=60, ns=4, nl=32)
    q = [c.q.cuda(), torch.flip(c.q, (0,)).contiguous().cuda()]
    steps, streams = [skv.Kv4Step(c.p, c.pool) for _ in q], [torch.cuda.Stream() for _ in q]
    want = [[x.clone() for x in (*s.attend_all(x), *s.run(x))] for s, x in zip(steps, q)]
    for s in steps:
        s.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, st in zip(steps, q, streams):
            s.attend_all(x, stream=st)
            s.run(x, stream=st)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert torch.equal(s.out, w[2]) and torch.equal(s.lse, w[3]) and int(s.status.item()) == 0


# ---------------------------------------------------------------------------- append


def assert_coded(got, y, tol, group):
    """(codes, s, z) of rows y known to tol: the step and centre within their roundings, each code one of
    the nearest to its entry under the stored step and centre (or the last one, for what lies outside).

    hi and lo are off by tol's largest in the group, their difference and sum by twice that, the
    fp32 arithmetic by 2^-22 of |lo| + |hi| besides."""
    c, s, z = got
    g = y.reshape(*y.shape[:-1], D // group, group)
    t = np.broadcast_to(tol, y.shape).reshape(g.shape).max(-1)
    lo, hi = g.min(-1), g.max(-1)
    t = t + 2.0 ** -22 * (np.abs(lo) + np.abs(hi))
    want = (hi - lo) / 15
    assert np.all(np.abs(s - want) <= HALF * want + t)
    mid = (hi + lo) / 2 + s / 2
    assert np.all(np.abs(z - mid) <= HALF * np.abs(mid) + 2 * t)
    err = np.abs(g - z[..., None] - s[..., None] * (c.reshape(g.shape).astype(np.float64) - 8))
    ends = ((c.reshape(g.shape) == 0) & (g <= z[..., None] - 8 * s[..., None])) | (
        (c.reshape(g.shape) == 15) & (g >= z[..., None] + 7 * s[..., None]))
    assert np.all(ends | (err <= s[..., None] / 2 + 2 * t[..., None]))
    assert np.all(err <= s[..., None] * (0.5 + 2.0 ** -5) + HALF * np.abs(z[..., None]) + 4 * t[..., None])


@pytest.mark.parametrize("n,H,G,dtype,group,bs,rot,style,norm,kw", [
    (1, 1, 1, "bf16", 32, 16, 128, 0, True, {}),
    (40, 2, 4, "bf16", 32, 16, 128, 0, True, {}),
    (40, 3, 16, "bf16", 64, 48, 64, 1, True, {}),
    (333, 8, 8, "bf16", 128, 32, 128, 1, False, {}),
    (40, 2, 5, "f32", 32, 16, 128, 0, True, {}),
    (700, 4, 3, "f32", 64, 64, 64, 1, True, {}),
    (40, 3, 2, "f32", 128, 16, 0, 0, False, {}),
    (60, 2, 4, "bf16", 32, 32, 128, 0, True, dict(host=0.5)),
    (60, 2, 4, "bf16", 64, 16, 128, 0, True, dict(host=0.4, per_head=True)),
    (60, 2, 4, "bf16", 32, 16, 128, 0, True, dict(part=64)),
])
def test_append(skv, n, H, G, dtype, group, bs, rot, style, norm, kw):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rng = np.random.default_rng(n)
    kw = dict(kw)
    part = kw.pop("part", D)
    B, span = 3, 2 * n + 40
    c = Case(skv, [span] * B, H, G, group=group, bs=bs, **kw)
    before = [[None if a is None else a.copy() for a in c.downloaded(kv)] for kv in range(2)]
    g = torch.Generator().manual_seed(n)
    row = torch.randn((n, H * G * D + 2 * H * D + 24), generator=g).to(dt)
    row[:, -24 - H * D:-24] *= 3.0
    q, k, v = (row[:, :H * G * D].view(n, H * G, D), row[:, H * G * D:(H * G + H) * D].view(n, H, D),
               row[:, (H * G + H) * D:(H * G + 2 * H) * D].view(n, H, D))
    gam = [(1 + 0.3 * torch.randn(part, generator=g)).to(dt) if norm else None for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
    # distinct (request, position) pairs, some tokens padding
    at = rng.permutation(B * span)[:n]
    req, pos = (at // span).astype(np.int32), (at % span).astype(np.int32)
    live = rng.random(n) < 0.85
    live[0] = True
    pos_in, req_in = np.where(live, pos, -1).astype(np.int32), np.where(rng.random(n) < 0.5, req, np.where(live, req, -1)).astype(np.int32)
    p = skv.Problem(**{**vars(c.p), "dtype": skv.SKV_DTYPE_F32 if dtype == "f32" else skv.SKV_DTYPE_BF16})
    cu = lambda x: None if x is None else x.cuda()  # noqa: E731
    r = skv.Rotary(cu(inv) if rot else None, rot_dim=rot, style=style, norm_dim=part, eps=1e-6, q_gamma=cu(gam[0]),
                   k_gamma=cu(gam[1]))
    step = skv.TokenStep(p, r, c.pool)
    dev = row.cuda()
    qd, kd, vd = (dev[:, :H * G * D].view(n, H * G, D), dev[:, H * G * D:(H * G + H) * D].view(n, H, D),
                  dev[:, (H * G + H) * D:(H * G + 2 * H) * D].view(n, H, D))
    q_out = torch.full((n, H * G, D), 5.0, dtype=dt, device="cuda")
    step.append(qd, kd, vd, _dev(pos_in), _dev(req_in), q_out=q_out)
    torch.cuda.synchronize()
    assert int(step.status.item()) == 0
    ref, tol = token_reference(q, gam[0], pos, inv, 0, rot, style, part, 1e-6)
    half = torch.finfo(dt).eps / 2
    err = np.abs(q_out.double().cpu().numpy() - ref)
    assert np.all(err[live] <= half * np.abs(ref[live]) + (1 + half) * tol[live] + 1e-37)
    assert torch.all(q_out[torch.from_numpy(~live)] == 5.0)
    kref, ktol = token_reference(k, gam[1], pos, inv, 0, rot, style, part, 1e-6)
    vref = v.double().numpy()
    for kv, (y, t) in enumerate(((kref, ktol), (vref, np.zeros_like(vref)))):
        after = c.downloaded(kv)
        for b in range(B):
            mine = live & (req == b)
            for h in range(H):
                if mine.any():
                    got = c.read(kv, b, h, pos[mine].astype(np.int64), *after)
                    assert_coded(got, y[mine, h], t[mine, h], group)
                    # the reference's own codes there, and every other byte of both tiers is as it was
                    on_gpu, e = c.place(b, h, pos[mine].astype(np.int64))
                    for on, cache, head, new, old in ((on_gpu, c.gpu[kv], 0 if c.per_head else h, after[0], before[kv][0]),
                                                      (~on_gpu, c.host[kv], h, after[1], before[kv][1])):
                        if on.any():
                            cells, rows = cache.cells(e[on], head, pos[mine][on].astype(np.int64))
                            a, o = new.reshape(-1, cache.cell), old.reshape(-1, cache.cell)
                            ng = D // group
                            for cl, rw in zip(cells, rows):
                                o[cl, 64 * rw:64 * rw + 64] = a[cl, 64 * rw:64 * rw + 64]
                                o[cl, 1024 + 4 * ng * rw:1024 + 4 * ng * (rw + 1)] = a[cl, 1024 + 4 * ng * rw:1024 + 4 * ng * (rw + 1)]
        for new, old in zip(after, before[kv]):
            assert (new is None) or np.array_equal(new, old)


def test_append_values_exact(skv):
    """V rows that 4 bits hold exactly come back as they are; rows of one value, of infinities and NaN."""
    rng = np.random.default_rng(2)
    c = Case(skv, [64], 1, 1)
    n = 40
    codes = rng.integers(0, 16, (n, D))
    codes[:, ::32], codes[:, 1::32] = 0, 15  # each group's ends
    v = torch.from_numpy(0.5 * (codes - 8.0) + 3.0).to(torch.bfloat16)
    v[1], v[2] = 2.5, 0.0
    v[3, 5], v[4, 40], v[5, 127] = float("inf"), float("nan"), float("-inf")
    v[6, :32] = torch.tensor([3.0e38, -3.0e38] * 16)
    r = skv.Rotary(None, rot_dim=0)
    step = skv.TokenStep(c.p, r, c.pool)
    at = torch.arange(n, dtype=torch.int32)
    step.append(None, v[:, None].cuda(), v[:, None].cuda(), at.cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"))
    p = skv.Problem(**{**vars(c.p), "n_local": 64, "dtype": skv.SKV_DTYPE_F32})
    for got in skv.Kv4Step(p, c.pool).gather():
        got = got[0, 0, :n].cpu()
        want = v.float()
        bad = torch.zeros((n, D), dtype=torch.bool)
        bad[3, :32] = bad[4, 32:64] = bad[5, 96:] = bad[6, :32] = True
        assert torch.all(torch.isnan(got[bad])) and torch.equal(got[~bad], want[~bad])


def test_append_refusals(skv):
    """Bad entries and positions: flagged, nothing written."""
    c = Case(skv, [64, 64], 2, 2)
    old = [c.pool.gpu_k.clone(), c.pool.gpu_v.clone()]
    c.pool.slot_table[0, 1] = c.pool.gpu_k.shape[0]
    c.pool.slot_table[1, 1] = -1
    step = skv.TokenStep(c.p, skv.Rotary(None, rot_dim=0), c.pool)
    k = torch.randn((4, 2, D)).to(torch.bfloat16).cuda()
    pos = torch.tensor([20, 20, 64, 5], dtype=torch.int32, device="cuda")
    req = torch.tensor([0, 1, 0, 2], dtype=torch.int32, device="cuda")
    step.append(None, k, k, pos, req)
    assert int(step.status.item()) == skv.SKV_DEV_BAD_SLOT | skv.SKV_DEV_BAD_LENGTH | skv.SKV_DEV_BAD_INDEX
    assert torch.equal(c.pool.gpu_k, old[0]) and torch.equal(c.pool.gpu_v, old[1])


@pytest.mark.parametrize("grown", [False, True])
def test_written_then_read(skv, grown):
    """The same rows written over and read back many times with nothing waiting between, and (grown) entries of a
    table that its own kernel moves every time: each read sees the write ahead of it on the stream."""
    B, H, G, bs, n = 24, 2, 4, 16, 24 * 16
    lens = torch.full((B,), 0 if grown else 16, dtype=torch.int32, device="cuda")
    p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=64, topk=0, n_sink=0, n_local=16,
                    block_size=bs, seq_lens=lens)
    table = torch.zeros((B, 4), dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B)
    pool = skv.Kv4Pool.empty(3 * B, H, bs, table)
    free = torch.arange(3 * B, dtype=torch.int32, device="cuda")
    tables = skv.BlockTables(p, table, free) if grown else None
    step = skv.Kv4Step(p, pool)
    tokens = skv.TokenStep(p, skv.Rotary(None, rot_dim=0), pool)
    at = torch.arange(16, dtype=torch.int32, device="cuda").repeat(B)
    req = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(16)
    q = torch.randn((B, H * G, D), device="cuda").to(torch.bfloat16)
    rows = [torch.randn((2, n, H, D), device="cuda").to(torch.bfloat16) for _ in range(30)]
    more, less = (torch.full((B,), x, dtype=torch.int32, device="cuda") for x in (16, -64))

    def once(x, waits):
        a, r = (at, req) if tables is None else tables.update(more, n)[:2]
        if waits:
            torch.cuda.synchronize()
        tokens.append(None, x[0], x[1], a, r)
        if waits:
            torch.cuda.synchronize()
        got = [*step.gather(), *(y.clone() for y in step.attend_all(q))]
        if waits:
            torch.cuda.synchronize()
        if tables is not None:
            tables.update(less)
            # the stack's top changes places with its bottom: the next blocks are others
            free.copy_(free.roll(5))
        return got

    want = [once(x, True) for x in rows]
    got = [once(x, False) for x in rows]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
    for x, g in zip(rows, got):  # a step of the 15th of a group's range at most, its halves' roundings on top
        for kv in range(2):
            y = x[kv].double().view(B, 16, H, D).transpose(1, 2)
            span = y.view(B, H, 16, 4, 32)
            tol = (span.amax(-1) - span.amin(-1)) / 15 * 0.6 + 2.0 ** -7 * span.abs().amax(-1)
            assert ((g[kv].double() - y).abs().view(span.shape) <= tol.unsqueeze(-1)).all()
    assert int(step.status.item()) == 0 and int(tokens.status.item()) == 0
