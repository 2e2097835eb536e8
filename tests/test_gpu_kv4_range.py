"""Attention over a cache in 4 bits whose value steps differ by orders of magnitude -- between the groups of a
row, between the rows of a history, between what one head attends and another -- against fp64 numpy."""

import numpy as np
import pytest
import torch

import kv4_ref
from test_gpu_kv4 import Case, _dev

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def attention(q, kv, vv, scale, count=None, adds=None):
    """(out, lse, tolerance of out, of lse) of rows that occur count times each (once), their sums of at most `adds`
    additions in turn (as many as rows, and 64), as kv4_ref.attention, but the fp16 operands held to what their own head
    and channel group needs.

    A weight times a step, w = p s, is fp16 under a power of two that keeps the largest w of its head and
    group at 2^7 at least: it is off by 2^-11 of itself (half a step) or, under the normal range, by half of
    2^-24, which is 2^-32 of that largest.  Codes are at most 15.  Where a unit's largest w has
    fallen under 2^-103 of the scale of 1 the power of two ends: 2^-25 of 2^-110 a key, over a sum of
    weights of 2^-28 at least.  A logit is off as kv4_ref.attention says, but counts by its own weight.  The
    other terms -- the sums' 2^-23 of their own group's parts, the output's rounding -- are kv4_ref.attention's."""
    k, v = kv4_ref.values(*kv), kv4_ref.values(*vv)
    rep = lambda a: np.repeat(np.abs(a), D // a.shape[-1], -1)  # noqa: E731
    count = np.ones(k.shape[0]) if count is None else count
    n = count.sum()
    adds = n + 64 if adds is None else adds
    x = scale * (q @ k.T)
    dx = scale * 160 * 2.0 ** -23 * (np.abs(q) @ (23 * rep(kv[1]) + rep(kv[2])).T)
    m = x[:, count > 0].max(-1, keepdims=True)
    p = np.where(count > 0, np.exp(np.minimum(x - m, 0)), 0)
    largest = (p[:, :, None] * rep(vv[1])[None, :, ::D // vv[1].shape[-1]]).max(1).repeat(D // vv[1].shape[-1], -1)
    p = p * count
    l = p.sum(-1, keepdims=True)
    out = p @ v / l
    part = 23 * rep(vv[1]) + rep(vv[2])
    rel = 2.0 ** -20 + adds * 2.0 ** -23
    off = (p * dx) @ part / l + (p * dx).sum(-1, keepdims=True) / l * np.abs(out)
    tol = (p @ (15 * rep(vv[1]))) / l * 2.0 ** -11 + rel * (p @ part) / l + off
    tol = tol + n * 15 * (2.0 ** -32 * largest / l + 2.0 ** (-25 - 110 + 28))
    lse = (m + np.log(l))[:, 0]
    return out, lse, tol + 2.0 ** -8 * np.abs(out), (p * dx).sum(-1) / l[:, 0] + rel + 2.0 ** -22 * np.abs(lse)


def check(c, out, lse, at=None):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, L in enumerate(c.lens):
        for h in range(c.H):
            heads = slice(h * c.G, (h + 1) * c.G)
            rows = np.arange(L) if at is None else np.array(at(b))
            ref, rl, tol, tl = attention(c.q[b, heads].double().numpy(), c.unit(0, b, h, rows), c.unit(1, b, h, rows), c.scale)
            err = np.abs(out[b, heads] - ref)
            assert np.all(err <= tol + 1e-37), (b, h, float((err / (tol + 1e-37)).max()))
            assert np.all(np.abs(lse[b, heads] - rl) <= tl), (b, h, np.abs(lse[b, heads] - rl).max(), tl)


def build(skv, G, group, k, v, q=None, listed=False):
    """A request of 900 rows a head, K and V rows k(rng, t), v(rng, t)."""
    n = 900
    c = Case(skv, [n], 2, G, group=group, **(dict(k=0, ns=4, nl=n - 4) if listed else {}))
    rng = np.random.default_rng(7)
    t = np.arange(n)
    for h in range(2):
        for kv, make in enumerate((k, v)):
            c.write(kv, 0, h, t, make(rng, t))
            c.rows[kv, 0, h] = c.read(kv, 0, h, t)
    if q is not None:
        c.q = torch.from_numpy(np.stack([q(rng, c.G) for _ in range(2)])).to(torch.bfloat16).reshape(1, 2 * G, D)
    c.upload()
    return c


def attend(c, listed):
    q = c.q.cuda()
    out, lse = c.step.attend(q) if listed else c.step.attend_all(q)
    first = out.clone(), lse.clone()
    again = c.step.attend(q) if listed else c.step.attend_all(q)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(c.step.status.item()) == 0
    check(c, *first)
    return first


def normal(rng, t):
    return rng.standard_normal((len(t), D))


def skewed(rng, t):
    """Values at the upper end of their groups but for one: codes that are lost move the output by half a group's range."""
    return np.where(np.arange(D) % 32 == 5, -1.0, 1.0) + 0.05 * rng.standard_normal((len(t), D))


U = np.where(np.arange(D) // 32 % 2, 1.0, -1.0)  # a direction of keys that their centres hold, not their steps


SHAPES = [(8, 32, False), (3, 64, False), (8, 128, False), (16, 32, False), (12, 128, False), (8, 32, True), (5, 64, True),
          (4, 128, True), (16, 64, True)]


@pytest.mark.parametrize("G,group,listed", SHAPES)
@pytest.mark.parametrize("apart", [10, 25, 35, 60])
def test_groups_apart(skv, G, group, listed, apart):
    """Groups of a row whose steps are 2^apart from each other: each keeps its own precision."""
    scale = np.exp2(-apart * (np.arange(D) // group % 4 == 1) + 10.0 * (np.arange(D) // 64 == 1))
    attend(build(skv, G, group, normal, lambda rng, t: skewed(rng, t) * scale, listed=listed), listed)


@pytest.mark.parametrize("G,group,listed", SHAPES)
@pytest.mark.parametrize("where", [0, 451, 899])
def test_row_that_no_head_attends(skv, G, group, listed, where):
    """One row of values 2^40 as large as the others', with a weight of 2^-90: the others are as without it."""

    def k(rng, t):
        x = 0.3 * normal(rng, t)
        x[where] = -8.0 * U
        return x

    def v(rng, t):
        x = skewed(rng, t)
        x[where] *= 2.0 ** 40
        return x

    attend(build(skv, G, group, k, v, lambda rng, g: 0.7 * U + 0.1 * rng.standard_normal((g, D)), listed), listed)


@pytest.mark.parametrize("G,group,listed", SHAPES)
def test_row_that_one_head_attends(skv, G, group, listed):
    """The same row all that every other head attends, and nothing to those between."""

    def k(rng, t):
        x = 0.3 * normal(rng, t)
        x[300] = 8.0 * U
        return x

    def v(rng, t):
        x = skewed(rng, t)
        x[300] *= 2.0 ** 40
        return x

    def q(rng, g):
        return np.where(np.arange(g) % 2, 0.7, -0.7)[:, None] * U + 0.1 * rng.standard_normal((g, D))

    attend(build(skv, G, group, k, v, q, listed), listed)


@pytest.mark.parametrize("G,group,listed", SHAPES)
@pytest.mark.parametrize("falling", [False, True])
def test_weights_against_steps(skv, G, group, listed, falling):
    """Logits that rise by 60 powers of two along the history while the steps fall by as many (or the other way
    round): every row has an equal part in the sum, whatever its weight or its step alone."""
    u = U * D ** -0.5
    at = lambda t: (t if falling else 899 - t) / 899.0 * 60  # noqa: E731

    def k(rng, t):
        return 0.05 * normal(rng, t) + (at(t) * np.log(2) * D ** 0.5 / 8)[:, None] * u

    def v(rng, t):
        return skewed(rng, t) * np.exp2(-at(t))[:, None]

    attend(build(skv, G, group, k, v, lambda rng, g: 8 * u + 0.1 * rng.standard_normal((g, D)), listed), listed)


@pytest.mark.parametrize("G,group,listed", SHAPES)
@pytest.mark.parametrize("e", [-110, -70, 60, 100, 118, 120, 125])
@pytest.mark.parametrize("kind", ["constant", "one group", "steps"])
def test_magnitudes(skv, G, group, listed, kind, e):
    """Values from the ends of fp32: groups of one value (steps of 0), one of them beside others, and steps themselves."""
    def v(rng, t):
        x = skewed(rng, t)
        if kind == "steps":
            return x * 2.0 ** e
        if kind == "one group":
            x[:, :group] = 1.5 * 2.0 ** e
            return x
        return np.full((len(t), D), -1.25 * 2.0 ** e)

    attend(build(skv, G, group, normal, v, listed=listed), listed)


@pytest.mark.parametrize("G,group,listed", SHAPES)
def test_heads_alone(skv, G, group, listed):
    """A head's bits are of its own query, whatever maxima and operands the heads beside it meet."""
    def v(rng, t):
        return skewed(rng, t) * np.exp2(rng.integers(-12, 12, (len(t), 1)))

    c = build(skv, G, group, normal, v, listed=listed)
    first = attend(c, listed)
    c.q[:, ::2] *= 40
    out, lse = attend(c, listed)
    assert torch.equal(out[:, 1::2], first[0][:, 1::2]) and torch.equal(lse[:, 1::2], first[1][:, 1::2])
    assert not torch.equal(out[:, ::2], first[0][:, ::2])
