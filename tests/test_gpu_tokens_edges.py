"""Norm and rotation at their edges."""

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


def _problem(skv, H, Hq, d, dtype, max_len=1 << 20, batch=1):
    return skv.Problem(batch=batch, n_kv_heads=H, n_q_heads=Hq, d_qk=d, d_v=d, max_len=max_len, topk=0, n_sink=0,
                       n_local=0, block_size=16, seq_lens=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                       dtype=skv.SKV_DTYPE_F32 if dtype == torch.float32 else skv.SKV_DTYPE_BF16)


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


PARTIAL = [
    # d, norm_dim, rot_start, rot_dim: the norm ends with the rotated span, inside it, before it, behind it
    (128, 64, 0, 64), (128, 32, 0, 64), (128, 40, 64, 32), (128, 96, 0, 32), (256, 128, 0, 128), (576, 512, 0, 64),
]


@pytest.mark.parametrize("style", ["half", "pair"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,nd,rs,rd", PARTIAL)
def test_a_row_whose_norm_is_nan_keeps_its_untouched_entries(skv, d, nd, rs, rd, dtype, style):
    """A NaN under the norm, or a normed part of zeros with eps 0, makes the factor NaN or infinite;
    entries outside the norm and the rotation are taken as they are all the same."""
    g = torch.Generator().manual_seed(d + nd + rs)
    q, k = (torch.randn((5, h, d), generator=g).to(dtype) for h in (6, 2))
    for x in (q, k):
        x[1, 0, 3] = float("nan")
        x[2, 1, :nd] = 0.0
        x[3, 0, nd - 1] = float("inf")
    inv = (10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)).float().cuda()
    gam = torch.ones(nd, dtype=dtype, device="cuda")
    rot = skv.Rotary(inv, rot_dim=rd, rot_start=rs, style=skv.SKV_ROPE_HALF if style == "half" else skv.SKV_ROPE_PAIR,
                     norm_dim=nd, eps=0.0, q_gamma=gam, k_gamma=gam)
    pos = torch.tensor([0, 5, 77, 1000, 9], dtype=torch.int32).cuda()
    out = skv.TokenStep(_problem(skv, 2, 6, d, dtype), rot).norm_rope(q.cuda(), k.cuda(), pos)
    e = torch.arange(d)
    plain = (e >= nd) & ((e < rs) | (e >= rs + rd))
    assert bool(plain.any())
    for got, x in zip(out, (q, k)):
        assert torch.equal(got.cpu()[..., plain], x[..., plain])
        assert bool(torch.isfinite(got.cpu()[[0, 4]]).all())


def _pi(bits):
    """pi * 2^bits by Machin's formula, in whole numbers."""
    def arctan_inv(x):
        total = term = (1 << (bits + 32)) // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    return (4 * (4 * arctan_inv(5) - arctan_inv(239))) >> 32


def _exact_cos_sin(t, f):
    """cos and sin of t * f with the angle reduced in 400-bit whole numbers."""
    bits = 400
    num, den = float(f).as_integer_ratio()
    two_pi = 2 * _pi(bits)
    ang = (t * num << bits) // den % two_pi
    if 2 * ang > two_pi:
        ang -= two_pi
    x = ang / 2 ** bits  # in [-pi, pi], rounded once
    return np.cos(x), np.sin(x)


@pytest.mark.parametrize("d", [128, 256])
def test_fast_frequencies_at_far_positions(skv, d):
    """Frequencies to 1,000 radians a position, of either sign, at positions to 2^31: the fp32 row
    (1, 0) turns into (cos, sin) of the exact angle.

    Bounds: 2^-22 for the functions; the reduced angle is at most an eighth of a turn and rounded to
    fp32, 2^-24 pi / 4; its turn is a fraction of 64 bits times a position below 2^31, off by at most
    2^-32 turns: together below 2^-21."""
    inv = torch.tensor([0.3, 0.75, 1.0, 2.0, 3.1, 5.5, 6.28, 6.2831855, 17.0, 99.5, 333.25, 1000.0, -0.4, -1.0, -5.0,
                        -123.5], dtype=torch.float32)
    inv = inv.repeat(d // 32)
    pos = [0, 1, 12345, 2 ** 24 + 1, 10 ** 9 + 7, 2 ** 30 - 1, 2 ** 31 - 3, 2 ** 31 - 2]
    x = torch.zeros((len(pos), 1, d))
    x[..., :d // 2] = 1.0
    rot = skv.Rotary(inv.cuda(), rot_dim=d)
    out, _ = skv.TokenStep(_problem(skv, 1, 1, d, torch.float32, max_len=2 ** 31 - 1), rot).norm_rope(
        x.cuda(), x.cuda(), torch.tensor(pos, dtype=torch.int32).cuda())
    for i, t in enumerate(pos):
        for j in range(16):
            c, s = _exact_cos_sin(t, float(inv[j]))
            assert abs(float(out[i, 0, j]) - c) <= 2.0 ** -21, (t, float(inv[j]))
            assert abs(float(out[i, 0, d // 2 + j]) - s) <= 2.0 ** -21, (t, float(inv[j]))


@pytest.mark.parametrize("d", [128, 576])
def test_padding_needs_no_request(skv, d):
    """A token of a negative position is padding whatever its request says, in both calls."""
    p = _problem(skv, 1, 2, d, torch.bfloat16, max_len=64, batch=2)
    n = 4
    q, k = (torch.randn((n, h, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda() for h in (2, 1))
    pool_k = torch.zeros((8, 1, 16, d), dtype=torch.bfloat16, device="cuda")
    pool = skv.Pool(pool_k, torch.zeros_like(pool_k), torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4))
    step = skv.TokenStep(p, skv.Rotary(None), pool)
    pos = torch.tensor([3, -1, -9, 5], dtype=torch.int32).cuda()
    req = torch.tensor([0, 2, 2 ** 31 - 1, 1], dtype=torch.int32).cuda()
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    step.norm_rope(q, k, pos, req, q_out=q_out, k_out=k_out)
    step.append(None, k, k, pos, req)
    assert int(step.status.item()) == 0
    live = torch.tensor([True, False, False, True])
    assert torch.equal(q_out[live], q[live]) and bool((q_out[~live] == 7.0).all())
    assert torch.equal(k_out[live], k[live]) and bool((k_out[~live] == 7.0).all())
    want = torch.zeros_like(pool_k)
    want[0, :, 3], want[4, :, 5] = k[0], k[3]
    assert torch.equal(pool_k, want)
    # a live token past the batch is an error still
    step.append(None, k, k, pos.abs(), req)
    assert int(step.status.item()) == skv.SKV_DEV_BAD_INDEX


@pytest.mark.parametrize("style", ["half", "pair"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rs,rd", [(128, 0, 0), (128, 32, 64), (256, 0, 128), (576, 512, 64)])
def test_untouched_entries_keep_their_bits(skv, d, rs, rd, dtype, style):
    """Zeros of either sign, the smallest and the largest numbers, infinities."""
    g = torch.Generator().manual_seed(d + rd)
    x = torch.randn((4, 3, d), generator=g).to(dtype)
    f = torch.finfo(dtype)
    special = torch.tensor([0.0, -0.0, f.tiny, -f.tiny, f.max, -f.max, float("inf"), -float("inf")]).to(dtype)
    x[1] = special.repeat(d // 8)
    inv = (10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / max(rd, 1))).float().cuda() if rd else None
    rot = skv.Rotary(inv, rot_dim=rd, rot_start=rs, style=skv.SKV_ROPE_HALF if style == "half" else skv.SKV_ROPE_PAIR)
    pos = torch.tensor([3, 5, 7, 11], dtype=torch.int32).cuda()
    _, got = skv.TokenStep(_problem(skv, 3, 3, d, dtype), rot).norm_rope(None, x.cuda(), pos)
    e = torch.arange(d)
    plain = (e < rs) | (e >= rs + rd)
    assert torch.equal(_bits(got.cpu()[..., plain]), _bits(x[..., plain]))
