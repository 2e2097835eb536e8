"""Norm and rotation at their edges."""

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
