"""Norm + rotation of new queries and keys, and their append to the pool, against fp64.

Tolerance, from the arithmetic: a row's mean square is a sum of fp32 squares with at most
NV * VE + 5 <= 45 roundings on any path, which the root halves (23 units of 2^-24); mean,
eps, root, reciprocal and two products add 7; cos and sin are within 2 units in the last
place (2^-22) plus the angle's own error; the turned pair adds 3 roundings.  Together under
48 * 2^-24 of |a| + |b|.  The angle's turn carries 2^-53 relative error: t * f * 2^-53.
Then one rounding of the result: half a step, eps / 2 of the value.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _inv(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


def reference(x, gamma, pos, inv, rot_start, rot_dim, style, norm_dim, eps):
    """(value, tolerance without the final rounding) in fp64 numpy; x [n, heads, d]."""
    x = x.double().numpy().copy()
    if gamma is not None:
        g = gamma.double().numpy()
        ms = (x[..., :norm_dim] ** 2).mean(-1, keepdims=True)
        x[..., :norm_dim] = x[..., :norm_dim] * g / np.sqrt(ms + eps)
    y, mag = x.copy(), np.abs(x)
    if rot_dim:
        i = np.arange(rot_dim // 2)
        ia, ib = (i, i + rot_dim // 2) if style == 0 else (2 * i, 2 * i + 1)
        ia, ib = ia + rot_start, ib + rot_start
        ang = pos.astype(np.float64)[:, None, None] * inv.double().numpy()
        c, s = np.cos(ang), np.sin(ang)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        m = np.abs(a) + np.abs(b)
        mag[..., ia] = mag[..., ib] = m
        far = np.zeros_like(mag)
        far[..., ia] = far[..., ib] = m * np.abs(ang) * 2.0 ** -53
    else:
        far = 0.0
    return y, 48 * 2.0 ** -24 * mag + far


def assert_rows(got, ref, tol):
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= half * np.abs(ref) + (1 + half) * tol + 1e-37), float((err - half * np.abs(ref) - tol).max())


CASES = [
    # n, H, Hq, d, dtype, rot_start, rot_dim, style, norm_dim, gammas
    (1, 1, 1, 128, "bf16", 0, 128, 0, 128, "qk"),
    (8, 8, 64, 128, "bf16", 0, 128, 0, 0, "qk"),
    (777, 2, 10, 128, "bf16", 0, 128, 1, 128, "k"),
    (33, 3, 21, 128, "bf16", 0, 64, 0, 128, ""),
    (33, 3, 21, 128, "bf16", 32, 96, 1, 64, "qk"),
    (19, 2, 14, 128, "bf16", 0, 16, 0, 128, "q"),
    (19, 2, 14, 128, "bf16", 0, 0, 0, 128, "qk"),
    (65, 4, 4, 128, "f32", 0, 128, 0, 128, "qk"),
    (65, 4, 12, 128, "f32", 64, 64, 1, 32, "qk"),
    (11, 1, 5, 64, "bf16", 0, 64, 0, 64, "qk"),
    (11, 2, 6, 96, "bf16", 0, 96, 0, 96, "qk"),
    (11, 2, 6, 96, "f32", 16, 80, 0, 96, "qk"),
    (11, 2, 6, 256, "bf16", 0, 256, 0, 256, "qk"),
    (11, 2, 6, 256, "f32", 0, 192, 0, 256, "qk"),
    (11, 1, 16, 576, "bf16", 512, 64, 1, 512, "k"),
    (11, 1, 16, 576, "bf16", 512, 64, 0, 512, "qk"),
    (11, 1, 4, 576, "f32", 8, 560, 0, 512, "qk"),
    (5, 1, 2, 1024, "bf16", 0, 1024, 0, 1024, "qk"),
    (5, 1, 2, 1024, "f32", 0, 1024, 0, 1024, "qk"),
    # a norm of a part of the row whose entries turn with entries outside it
    (33, 3, 21, 128, "bf16", 0, 128, 0, 64, "qk"),
    (21, 2, 6, 128, "f32", 0, 128, 0, 40, "k"),
    (700, 2, 6, 256, "bf16", 32, 192, 0, 104, "q"),
    # more rows a token than a stage holds
    (350, 16, 144, 256, "bf16", 0, 256, 0, 192, "qk"),
    (320, 8, 200, 128, "f32", 0, 128, 1, 128, "qk"),
]


def _make(skv, case, seed=1, max_len=1 << 20):
    n, H, Hq, d, dt, rs, rd, style, nd, gs = case
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = _gen(seed)
    fused = torch.randn((n, (Hq + H) * d + 16), generator=g).to(dtype)
    q, k = fused[:, :Hq * d].view(n, Hq, d), fused[:, Hq * d:(Hq + H) * d].view(n, H, d)
    gam = {s: (1 + 0.3 * torch.randn(nd or d, generator=g)).to(dtype) if s in gs else None for s in "qk"}
    pos = torch.randint(0, max_len, (n,), generator=g).to(torch.int32)
    inv = _inv(rd)
    p = skv.Problem(batch=1, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=d, max_len=max_len, topk=0, n_sink=0, n_local=0,
                    block_size=16, seq_lens=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    dtype=skv.SKV_DTYPE_F32 if dt == "f32" else skv.SKV_DTYPE_BF16)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    r = skv.Rotary(cu(inv) if rd else None, rot_dim=rd, rot_start=rs, style=style, norm_dim=nd, eps=1e-5,
                   q_gamma=cu(gam["q"]), k_gamma=cu(gam["k"]))
    return p, r, fused, q, k, gam, pos, inv


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("max_len", [1 << 20, 2 ** 31 - 1])
def test_norm_rope(skv, case, max_len):
    p, r, fused, q, k, gam, pos, inv = _make(skv, case, max_len=max_len)
    n, H, Hq, d, dt, rs, rd, style, nd, gs = case
    pos[0], pos[-1] = 0, max_len - 1
    dev = fused.cuda()
    qd, kd = dev[:, :Hq * d].view(n, Hq, d), dev[:, Hq * d:(Hq + H) * d].view(n, H, d)
    step = skv.TokenStep(p, r)
    q_out, k_out = step.norm_rope(qd, kd, pos.cuda())
    for got, x, s in ((q_out, q, "q"), (k_out, k, "k")):
        ref, tol = reference(x, gam[s], pos.numpy(), inv, rs, rd, style, nd or d, 1e-5)
        assert_rows(got, ref, tol)
    assert torch.equal(dev.cpu(), fused)  # the inputs stay
    # in place at the fused rows' stride: the same bits, and nothing beside them
    tail = dev[:, (Hq + H) * d:].clone()
    a, b = step.norm_rope(qd, kd, pos.cuda(), q_out=qd, k_out=kd)
    assert a is qd and b is kd and torch.equal(qd, q_out) and torch.equal(kd, k_out)
    assert torch.equal(dev[:, (Hq + H) * d:], tail)
    # one side alone
    only, none = step.norm_rope(None, k.cuda(), pos.cuda())
    assert only is None and torch.equal(none, k_out)
    assert int(step.status.item()) == 0


def test_rotation_keeps_angles_of_far_positions(skv):
    """Positions whose fp32 angle is off by whole radians: fp32 rows turned by the exact angle."""
    case = (7, 1, 1, 128, "f32", 0, 128, 0, 128, "")
    p, r, fused, q, k, gam, pos, inv = _make(skv, case, max_len=2 ** 31 - 1)
    pos[:] = torch.tensor([0, 1, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 30 - 1, 2 ** 31 - 3, 2 ** 31 - 2], dtype=torch.int32)
    x = torch.zeros((7, 1, 128))
    x[..., :64] = 1.0  # the pairs become (cos, sin)
    out, _ = skv.TokenStep(p, r).norm_rope(x.cuda(), x.cuda(), pos.cuda())
    ang = pos.double().numpy()[:, None] * inv.double().numpy()
    want = np.concatenate([np.cos(ang), np.sin(ang)], -1)
    # 2^-22 of the functions, 2^-25 of the reduced angle and t f 2^-53 of the turn
    assert np.all(np.abs(out[:, 0].double().cpu().numpy() - want) <= 2.0 ** -21 + 2 * np.concatenate([ang, ang], -1) * 2.0 ** -53)


def test_padding_and_bad_tokens_write_nothing(skv):
    case = (6, 2, 4, 128, "bf16", 0, 128, 0, 128, "qk")
    p, r, fused, q, k, gam, pos, inv = _make(skv, case, max_len=1000)
    step = skv.TokenStep(p, r)
    qd, kd = q.cuda().contiguous(), k.cuda().contiguous()
    fill = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    full, _ = step.norm_rope(qd, kd, torch.tensor([5, 5, 5, 5, 999, 0], dtype=torch.int32).cuda())
    for ids, posn, live, bits in [
        (None, [5, -1, 5, -7, 999, 0], [1, 0, 1, 0, 1, 1], 0),
        (None, [5, 1000, 5, 5, 999, 0], [1, 0, 1, 1, 1, 1], skv.SKV_DEV_BAD_LENGTH),
        ([0, 0, -1, 0, 0, 0], [5, 5, 5, 5, 999, 0], [1, 1, 0, 1, 1, 1], 0),
        ([0, 0, 0, 1, 0, 0], [5, 5, 5, 5, 999, 0], [1, 1, 1, 0, 1, 1], skv.SKV_DEV_BAD_INDEX),
    ]:
        step.status.zero_()
        got, _ = step.norm_rope(qd, kd, torch.tensor(posn, dtype=torch.int32).cuda(),
                                None if ids is None else torch.tensor(ids, dtype=torch.int32).cuda(),
                                q_out=fill(qd), k_out=fill(kd))
        for i, on in enumerate(live):
            assert torch.equal(got[i], full[i] if on else fill(qd)[i]), i
        assert int(step.status.item()) == bits


def test_rows_of_zeros_and_nonfinite_rows_stay_apart(skv):
    case = (4, 1, 2, 128, "bf16", 0, 128, 0, 128, "qk")
    p, r, fused, q, k, gam, pos, inv = _make(skv, case)
    q = q.contiguous()
    step = skv.TokenStep(p, r)
    clean, _ = step.norm_rope(q.cuda(), k.cuda(), pos.cuda())
    q[1, 0], q[2, 1, 5], q[3, 0, 9] = 0.0, float("inf"), float("nan")
    got, _ = step.norm_rope(q.cuda(), k.cuda(), pos.cuda())
    assert torch.count_nonzero(got[1, 0]) == 0
    assert torch.isnan(got[3, 0]).all()
    for i, h in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 1)):
        assert torch.equal(got[i, h], clean[i, h])


# ---------------------------------------------------------------------------- append

APPEND = [
    # B, H, Hq, d, dv, dtype, bs, latent, table_heads, host
    (4, 2, 8, 128, 128, "bf16", 16, False, 0, False),
    (4, 2, 8, 128, 128, "bf16", 16, False, 0, True),
    (3, 4, 20, 128, 128, "bf16", 16, False, 1, False),
    (3, 4, 20, 128, 128, "bf16", 16, False, 1, True),
    (2, 2, 6, 128, 128, "f32", 16, False, 0, False),
    (2, 1, 3, 128, 64, "bf16", 1, False, 0, False),
    (2, 2, 2, 64, 128, "f32", 7, False, 0, False),
    (3, 1, 16, 576, 512, "bf16", 1, True, 0, False),
    (3, 1, 16, 576, 512, "bf16", 16, True, 0, True),
]


def _pool(skv, spec, cap, seed):
    """Pools filled with noise, a random table (negative entries: host blocks)."""
    B, H, Hq, d, dv, dt, bs, latent, heads, host = spec
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = _gen(seed)
    per = (cap + bs - 1) // bs
    rows = B * (H if heads else 1)
    shape = lambda n, w: (n, bs, w) if heads else (n, H, bs, w)  # noqa: E731
    n = rows * per + 3
    gk = torch.randn(shape(n, d), generator=g).to(dtype)
    gv = None if latent else torch.randn(shape(n, dv), generator=g).to(dtype)
    table = torch.randperm(n, generator=g)[:rows * per].to(torch.int32).view((B, H, per) if heads else (B, per))
    hk = hv = None
    if host:
        nh = B * per + 2
        hk = torch.randn((nh, H, bs, d), generator=g).to(dtype)
        hv = None if latent else torch.randn((nh, H, bs, dv), generator=g).to(dtype)
        perm = torch.randperm(nh, generator=g)[:B * per].to(torch.int32).view(B, per)
        to_host = torch.rand(table.shape, generator=g) < 0.4
        hostent = -(perm[:, None].expand_as(table) if heads else perm) - 1
        table = torch.where(to_host, hostent, table)
    return gk, gv, table.contiguous(), hk, hv


def _expect(spec, k, v, pos, req, gk, gv, table, hk, hv):
    """Copies of the pools with every live token's rows put in place (K in fp64 beside its mask)."""
    B, H, Hq, d, dv, dt, bs, latent, heads, host = spec
    outs = [None if t is None else t.double().numpy().copy() for t in (gk, gv, hk, hv)]
    touched = [None if t is None else np.zeros(t.shape, bool) for t in (gk, gv, hk, hv)]
    for i in range(len(pos)):
        if pos[i] < 0 or req[i] < 0:
            continue
        for h in range(H):
            e = int(table[req[i], h, pos[i] // bs]) if heads else int(table[req[i], pos[i] // bs])
            off = int(pos[i] % bs)
            at = ((e, off) if heads else (e, h, off)) if e >= 0 else (-e - 1, h, off)
            for j, x in ((0, k), (1, v)):
                j = j if e >= 0 else j + 2
                if outs[j] is not None:
                    outs[j][at] = x[i, h]
                    touched[j][at] = True
    return outs, touched


def _check_pools(spec, got, before, outs, touched, tols):
    for j, (g, b4) in enumerate(zip(got, before)):
        if g is None:
            continue
        g = g.cpu()
        m = torch.from_numpy(touched[j])
        assert torch.equal(g[~m], b4[~m])  # rows that no token names
        if j % 2 == 1:  # V: the bits
            assert np.array_equal(g.double().numpy()[touched[j]], outs[j][touched[j]])
        else:
            err = np.abs(g.double().numpy() - outs[j])[touched[j]]
            half = torch.finfo(g.dtype).eps / 2
            assert np.all(err <= half * np.abs(outs[j][touched[j]]) + (1 + half) * tols)


@pytest.mark.parametrize("spec", APPEND)
@pytest.mark.parametrize("decode", [True, False])
def test_append(skv, spec, decode):
    B, H, Hq, d, dv, dt, bs, latent, heads, host = spec
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    cap = 75
    gk, gv, table, hk, hv = _pool(skv, spec, cap, 3)
    g = _gen(4)
    if decode:
        lens = torch.tensor([cap, 1, 0, 33][:B], dtype=torch.int32)
        n, pos, req = B, (lens - 1).numpy(), np.arange(B)
        posd = reqd = None
    else:
        lens = torch.zeros(B, dtype=torch.int32)
        pairs = [(b, t) for b in range(B) for t in range(0, cap, 1 + b)]
        order = torch.randperm(len(pairs), generator=g).tolist()
        pairs = [pairs[i] for i in order] + [(0, -1), (-1, 3), (-5, -5)]
        n, req, pos = len(pairs), np.array([b for b, _ in pairs]), np.array([t for _, t in pairs])
        posd, reqd = (torch.from_numpy(a).to(torch.int32).cuda() for a in (pos, req))
    row = torch.randn((n, (Hq + H) * d + H * dv), generator=g).to(dtype)
    q, k = row[:, :Hq * d].view(n, Hq, d), row[:, Hq * d:(Hq + H) * d].view(n, H, d)
    v = None if latent else row[:, (Hq + H) * d:].view(n, H, dv)
    rd, rs, nd = (64, 512, 512) if d == 576 else (d, 0, d)
    gam = (1 + 0.3 * torch.randn(nd, generator=g)).to(dtype)
    inv = _inv(rd)
    p = skv.Problem(batch=B, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=dv, max_len=cap, topk=0, n_sink=0, n_local=0,
                    block_size=bs, seq_lens=lens.cuda(), dtype=skv.SKV_DTYPE_F32 if dt == "f32" else skv.SKV_DTYPE_BF16)
    pin = lambda t: None if t is None else t.clone().pin_memory()  # noqa: E731
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    pool = skv.Pool(cu(gk), cu(gv), table.cuda(), pin(hk), pin(hv), table_heads=heads)
    r = skv.Rotary(inv.cuda(), rot_dim=rd, rot_start=rs, norm_dim=nd, q_gamma=None, k_gamma=gam.cuda())
    step = skv.TokenStep(p, r, pool)
    rowd = row.cuda()
    qd, kd = rowd[:, :Hq * d].view(n, Hq, d), rowd[:, Hq * d:(Hq + H) * d].view(n, H, d)
    vd = None if latent else rowd[:, (Hq + H) * d:].view(n, H, dv)
    q_out = torch.full((n, Hq, d), 3.0, dtype=dtype, device="cuda")
    step.append(qd, kd, vd, posd, reqd, q_out=q_out)
    torch.cuda.synchronize()
    assert int(step.status.item()) == 0
    live = (pos >= 0) & (req >= 0)
    refq, tolq = reference(q, None, pos, inv, rs, rd, 0, nd, 1e-6)
    assert_rows(q_out[torch.from_numpy(live)], refq[live], tolq[live])
    assert bool((q_out[torch.from_numpy(~live)] == 3.0).all())
    refk, tolk = reference(k, gam, pos, inv, rs, rd, 0, nd, 1e-6)
    before = (gk, gv, hk, hv)
    outs, touched = _expect(spec, refk, None if latent else v.double().numpy(), pos, req, gk, gv, table, hk, hv)
    _check_pools(spec, (pool.gpu_k, pool.gpu_v, pool.host_k, pool.host_v), before, outs, touched, tolk[live].max())
    # without queries: the same pool rows again
    again = skv.Pool(cu(gk), cu(gv), table.cuda(), pin(hk), pin(hv), table_heads=heads)
    assert skv.TokenStep(p, r, again).append(None, kd, vd, posd, reqd) is None
    torch.cuda.synchronize()
    assert torch.equal(again.gpu_k, pool.gpu_k)
    if hk is not None:
        assert torch.equal(again.host_k, pool.host_k)


def test_append_bad_entries_and_requests(skv):
    spec = (3, 2, 4, 128, 128, "bf16", 16, False, 0, False)
    gk, gv, table, _, _ = _pool(skv, spec, 64, 5)
    table[0, 1], table[1, 0] = gk.shape[0], -1  # past the pool; a host block without a host pool
    k = torch.randn((4, 2, 128), generator=_gen(6)).to(torch.bfloat16).cuda()
    p = skv.Problem(batch=3, n_kv_heads=2, n_q_heads=4, d_qk=128, d_v=128, max_len=64, topk=0, n_sink=0, n_local=0,
                    block_size=16, seq_lens=torch.tensor([70, -2, 64], dtype=torch.int32).cuda())
    r = skv.Rotary(None)
    for pos, req, bits, rows in [
        ([16, 0, 5, 63], [0, 1, 2, 2], skv.SKV_DEV_BAD_SLOT, [2, 3]),
        ([0, 64, 5, 63], [0, 2, 2, 3], skv.SKV_DEV_BAD_LENGTH | skv.SKV_DEV_BAD_INDEX, [0, 2]),
    ]:
        pool = skv.Pool(gk.cuda(), gv.cuda(), table.cuda())
        step = skv.TokenStep(p, r, pool)
        step.append(None, k, k, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(req, dtype=torch.int32).cuda())
        want = gk.clone()
        for i in rows:
            want[int(table[req[i], pos[i] // 16]), :, pos[i] % 16] = k[i].cpu()
        assert torch.equal(pool.gpu_k.cpu(), want)
        assert int(step.status.item()) == bits
    # positions from the lengths: one past the capacity and one below zero are flagged and skipped
    pool = skv.Pool(gk.cuda(), gv.cuda(), table.cuda())
    step = skv.TokenStep(p, r, pool)
    step.append(None, k[:3], k[:3])
    want = gk.clone()
    want[int(table[2, 3]), :, 15] = k[2].cpu()
    assert torch.equal(pool.gpu_k.cpu(), want)
    assert int(step.status.item()) == skv.SKV_DEV_BAD_LENGTH


def test_append_in_a_graph_and_on_another_stream(skv):
    """A captured append replays on new contents of its tensors; a call on a side stream lands there."""
    spec = (4, 2, 8, 128, 128, "bf16", 16, False, 0, False)
    gk, gv, table, _, _ = _pool(skv, spec, 64, 7)
    lens = torch.tensor([5, 17, 64, 1], dtype=torch.int32).cuda()
    p = skv.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=64, topk=0, n_sink=0, n_local=0,
                    block_size=16, seq_lens=lens)
    r = skv.Rotary(_inv(128).cuda(), rot_dim=128)
    g = _gen(8)
    new = lambda: [torch.randn((4, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (8, 2, 2)]  # noqa: E731
    q, k, v = new()
    pool = skv.Pool(gk.cuda(), gv.cuda(), table.cuda())
    step = skv.TokenStep(p, r, pool)
    q_out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.append(q, k, v, q_out=q_out)
    for it in range(2):
        q2, k2, v2 = new()
        q.copy_(q2), k.copy_(k2), v.copy_(v2)
        if it:
            lens.sub_(1)  # the last request becomes empty: padding
        graph.replay()
        other = skv.Pool(pool.gpu_k.clone(), pool.gpu_v.clone(), table.cuda())
        want_k = gk.cuda() if it == 0 else None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fresh = skv.Pool((want_k if want_k is not None else other.gpu_k).clone(), gv.cuda().clone(), table.cuda())
            got = skv.TokenStep(p, r, fresh).append(q, k, v)
        torch.cuda.current_stream().wait_stream(side)
        n = 4 if it == 0 else 3
        assert torch.equal(got[:n], q_out[:n])
        assert torch.equal(fresh.gpu_k, pool.gpu_k)
    assert int(step.status.item()) == 0


def test_no_token_and_one_token(skv):
    """Empty tensors do nothing; a lone token's stride has no meaning and is not looked at."""
    p, r, fused, q, k, gam, pos, inv = _make(skv, (2, 2, 4, 128, "bf16", 0, 128, 0, 0, "qk"))
    step = skv.TokenStep(p, r)
    n0 = skv.lib().skv_launch_count()
    none = lambda h: torch.zeros((0, h, 128), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    a, b = step.norm_rope(none(4), none(2), torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128) and skv.lib().skv_launch_count() == n0
    want = step.norm_rope(q.cuda().contiguous(), k.cuda().contiguous(), pos.cuda())
    odd = [x[:1].cuda().as_strided((1, x.shape[1], 128), (13, 128, 1)) for x in (q.contiguous(), k.contiguous())]
    got = step.norm_rope(*odd, pos[:1].cuda())
    assert torch.equal(got[0], want[0][:1]) and torch.equal(got[1], want[1][:1])
    got = step.norm_rope(*odd, pos[:1].cuda(), q_out=odd[0], k_out=odd[1])
    assert torch.equal(got[0], want[0][:1]) and torch.equal(got[1], want[1][:1])


def test_refuses_what_is_not_on_the_gpu(skv):
    p, r, fused, q, k, gam, pos, inv = _make(skv, (2, 2, 4, 128, "bf16", 0, 128, 0, 0, "qk"))
    step, n0 = skv.TokenStep(p, r), skv.lib().skv_launch_count()
    for args in ((q, k, pos.cuda()), (q.cuda(), k, pos.cuda()), (q.cuda(), k.cuda(), pos)):
        with pytest.raises(ValueError):
            step.norm_rope(*args)
    with pytest.raises(ValueError):
        step.norm_rope(q.cuda(), k.cuda(), pos.cuda(), q_out=torch.empty_like(q.contiguous()))
    assert skv.lib().skv_launch_count() == n0


def test_a_given_stream(skv):
    """Calls on a stream that is not the current one, their outputs theirs: freed ones are not handed
    to the current stream's work while the call may still write them."""
    p, r, fused, q, k, gam, pos, inv = _make(skv, (777, 8, 64, 128, "bf16", 0, 128, 0, 0, "qk"))
    step, side = skv.TokenStep(p, r), torch.cuda.Stream()
    qd, kd, posd = q.cuda(), k.cuda(), pos.cuda()
    want = step.norm_rope(qd, kd, posd)
    torch.cuda.synchronize()
    for _ in range(20):
        step.norm_rope(qd, kd, posd, stream=side)  # outputs dropped at once
        mine = torch.full_like(want[0], 3.0)
        assert bool((mine == 3.0).all())
    got = step.norm_rope(qd, kd, posd, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
