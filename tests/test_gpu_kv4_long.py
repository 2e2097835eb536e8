"""The cache in 4 bits over histories and lists of millions of keys -- tens and hundreds of tiles a warp -- against fp64
numpy: a table that repeats the blocks of a small pool, so that the rows that occur are few and counted."""

import numpy as np
import pytest
import torch

import kv4_ref
from test_gpu_kv4_range import U, attention

pytestmark = pytest.mark.gpu

D = 128
BLOCKS = 700


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def rows(kind, rng, bs, kv):
    """The rows of the pool's blocks, one head's K or V.  Levels: powers of two that a block's logits stand above the
    first one's; along the table they rise (or fall) by 60 and start again."""
    n = BLOCKS * bs
    at = np.arange(BLOCKS) / (BLOCKS - 1.0) * 60
    level = {"rising": at, "falling": at[::-1], "against": at, "spread": rng.permutation(at), "plain": 0 * at}[kind]
    level = np.repeat(level, bs)[:, None]
    x = rng.standard_normal((n, D))
    if kv == 0:
        return (0.3 if kind == "plain" else 0.05) * x + level * (np.log(2) * D ** 0.5 / (8 * D ** 0.5)) * U
    x = x * (0.25 + rng.random((n, 1))) + 0.3 * rng.standard_normal(D)
    return x * np.exp2(-level) if kind == "against" else x * np.exp2(rng.integers(-20, 20, (n, 1))) if kind == "spread" else x


class Long:
    def __init__(self, skv, lens, H, G, group, bs=16, kind="plain", agg=0, k=0, ns=0, nl=0, seed=1):
        self.skv, self.lens, self.H, self.G, self.bs = skv, lens, H, G, bs
        self.rng = rng = np.random.default_rng(seed)
        max_len = max(lens)
        per = -(-max_len // bs)
        # blocks in order, so that a level rises along every warp's walk
        self.table = np.stack([(np.arange(per) + 100 * b) % BLOCKS for b in range(len(lens))]).astype(np.int32)
        self.values, pools = {}, []
        for kv in range(2):
            cache = kv4_ref.Cache(BLOCKS, H, bs, group, rng)
            r = np.arange(BLOCKS * bs)
            for h in range(H):
                cache.put(r // bs, h, r % bs, rows(kind, rng, bs, kv))
                self.values[kv, h] = cache.raw(r // bs, h, r % bs)
            pools.append(torch.from_numpy(cache.pool).cuda())
        q = 0.1 * rng.standard_normal((len(lens), H * G, D)) + 8 * U * D ** -0.5
        if kind == "plain":
            q = rng.standard_normal((len(lens), H * G, D))
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        self.p = skv.Problem(batch=len(lens), n_kv_heads=H, n_q_heads=H * G, d_qk=D, d_v=D, max_len=max_len, topk=k,
                             n_sink=ns, n_local=nl, block_size=bs, seq_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                             group_agg=agg)
        self.step = skv.Kv4Step(self.p, skv.Kv4Pool(*pools, torch.from_numpy(self.table).cuda(), group=group))

    def row(self, b, at):
        """The pool's rows at positions of request b."""
        return self.table[b, at // self.bs].astype(np.int64) * self.bs + at % self.bs

    def count(self, b, at):
        return np.bincount(self.row(b, at), minlength=BLOCKS * self.bs).astype(np.float64)

    def tiles(self, keys, warps):
        """Tiles of a warp at the most, of `warps` warps a SM that share the keys of all units."""
        return keys / 16 / (warps * torch.cuda.get_device_properties(0).multi_processor_count) + 2

    def check(self, out, lse, counts, warps):
        """Sums: a tile is 17 additions of a warp, 16 warps a CTA and 304 CTAs follow."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        keys = sum(c.sum() for c in counts.values())
        tiles = self.tiles(keys, warps)
        assert self.tiles(keys, 16) > 64
        for (b, h), n in counts.items():
            hs = slice(h * self.G, (h + 1) * self.G)
            if n.sum() == 0:
                assert np.all(out[b, hs] == 0) and np.all(np.isneginf(lse[b, hs]))
                continue
            ref, rl, tol, tl = attention(self.q[b, hs].double().numpy(), self.values[0, h], self.values[1, h], D ** -0.5, n,
                                         17 * tiles + 400)
            err = np.abs(out[b, hs] - ref)
            assert np.all(err <= tol + 1e-37), (b, h, float((err / (tol + 1e-37)).max()))
            assert np.all(np.abs(lse[b, hs] - rl) <= tl), (b, h, np.abs(lse[b, hs] - rl).max(), tl)
        assert int(self.step.status.item()) == 0
        return out


SHAPES = [(8, 32, 16), (4, 64, 48), (3, 128, 32), (16, 32, 16), (12, 64, 16), (9, 128, 80)]


@pytest.mark.parametrize("kind", ["plain", "rising", "falling", "against", "spread"])
@pytest.mark.parametrize("G,group,bs", SHAPES)
def test_attend_all(skv, G, group, bs, kind):
    c = Long(skv, [1300003, 0, 5, 171717], 2, G, group, bs, kind)
    out, lse = (x.clone() for x in c.step.attend_all(c.q.cuda()))
    c.check(out, lse, {(b, h): c.count(b, np.arange(L)) for b, L in enumerate(c.lens) for h in range(2)}, 8)
    again = c.step.attend_all(c.q.cuda())
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_long_sums(skv, group):
    """Hundreds of tiles a warp, 1.9 million keys of 8 heads: what the tensor core truncates is not seen in the output.

    Rounded to bf16 an output is off by 2^-8 of itself at most, and so is their norm.  The sums stay about zero (codes
    against their complements): a warp's 8,000 additions are each off by 2^-23 of a sum of about 90 keys' parts,
    together 2^-16 of a part or 2^-12 of the output; one-sided sums would lose 1 % of it here."""
    L = 1900000
    c = Long(skv, [L], 8, 4, group)
    assert c.tiles(8 * L, 16) > 350
    out, lse = c.step.attend_all(c.q.cuda())
    counts = {(0, h): c.count(0, np.arange(L)) for h in range(8)}
    out = c.check(out, lse, counts, 12)
    ref = np.concatenate([attention(c.q[0, 4 * h:4 * h + 4].double().numpy(), c.values[0, h], c.values[1, h], D ** -0.5,
                                    counts[0, h])[0] for h in range(8)])
    assert np.linalg.norm(out[0] - ref) <= (2.0 ** -8 + 2.0 ** -10) * np.linalg.norm(ref)


@pytest.mark.parametrize("kind", ["plain", "rising", "against", "spread"])
@pytest.mark.parametrize("G,group,bs,agg", [(8, 32, 16, 0), (4, 64, 48, 0), (3, 128, 32, 0), (16, 32, 16, 0), (2, 64, 16, 2)])
def test_attend_list(skv, G, group, bs, agg, kind):
    k, L = (1400000, 1600000) if agg == 0 else (700000, 1600000)
    c = Long(skv, [L, 900], 2, G, group, bs, kind, agg=agg, k=k, ns=4, nl=100)
    heads = 2 * G if agg == 2 else 2
    idx = np.full((2, heads, k), -1, np.int32)
    lists = {}
    for b, n in enumerate(c.lens):
        for r in range(heads):
            some = np.sort(c.rng.permutation(n - 104)[:k] + 4)
            idx[b, r, :len(some)] = some
            lists[b, r] = np.concatenate([np.arange(4), some, np.arange(n - 100, n)])
    out, lse = c.step.attend(c.q.cuda(), torch.from_numpy(idx).cuda())
    if agg == 0:
        c.check(out, lse, {at: c.count(at[0], x) for at, x in lists.items()}, 8)
        return
    # a query head's own list: its head alone
    c.G, c.values = 1, {(kv, r): c.values[kv, r // G] for kv in range(2) for r in range(heads)}
    c.check(out, lse, {at: c.count(at[0], x) for at, x in lists.items()}, 8)


@pytest.mark.parametrize("agg", [0, 1, 2])
@pytest.mark.parametrize("G,group,bs", [(4, 32, 16), (8, 64, 48), (3, 128, 80), (16, 32, 32)])
def test_score(skv, G, group, bs, agg):
    """Tolerances as test_gpu_kv4.assert_scores, of the pool's rows."""
    L, ns, nl = 1600001, 19, 77
    c = Long(skv, [L, 33], 2, G, group, bs, agg=agg, ns=ns, nl=nl)
    assert c.tiles(2 * L, 16) > 64
    scores = torch.full((2, 2 * G if agg == 2 else 2, L), 7.0, device="cuda")
    c.step.score(c.q.cuda(), scores)
    at = c.row(0, np.arange(ns, L - nl))
    for h in range(2):
        qh = c.q[0, h * G:(h + 1) * G].double().numpy()
        k, s, z = c.values[0, h]
        rep = lambda a: np.repeat(np.abs(a), group, -1)  # noqa: E731
        x, m = qh @ kv4_ref.values(k, s, z).T, np.abs(qh) @ (23 * rep(s) + rep(z)).T
        if agg == 0:
            x, m = x.mean(0, keepdims=True), m.mean(0, keepdims=True)
        elif agg == 1:
            x, m = x.max(0, keepdims=True), m.max(0, keepdims=True)
        got = scores[0, h * G:(h + 1) * G] if agg == 2 else scores[0, h:h + 1]
        got = got.double().cpu().numpy()
        err = np.abs(got[:, ns:L - nl] - x[:, at])
        assert np.all(err <= (160 + 2 * G) * 2.0 ** -23 * m[:, at]), float((err / m[:, at]).max() * 2 ** 23)
        assert np.all(got[:, :ns] == 7) and np.all(got[:, L - nl:] == 7)
    assert torch.all(scores[1] == 7) and int(c.step.status.item()) == 0
