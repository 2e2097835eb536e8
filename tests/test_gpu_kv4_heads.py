"""The append in 4 bits for odd counts of KV heads: half of a warp then holds no row."""

import pytest
import torch

import kv4_ref

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def skv():
    import __graft_entry__

    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def append(skv, H, n, scale):
    """(values of V's rows, the rows) of n tokens of H heads, K and V of this scale."""
    bs, g = 16, torch.Generator().manual_seed(H)
    table = torch.arange(n // bs, dtype=torch.int32, device="cuda")[None].contiguous()
    p = skv.Problem(batch=1, n_kv_heads=H, n_q_heads=8 * H, d_qk=D, d_v=D, max_len=n, topk=0, n_sink=0, n_local=n,
                    block_size=bs, seq_lens=torch.full((1,), n, dtype=torch.int32, device="cuda"))
    pool = skv.Kv4Pool.empty(n // bs, H, bs, table)
    step = skv.TokenStep(p, skv.Rotary(None, rot_dim=0), pool)
    rows = torch.randn((n, 10 * H, D), generator=g).to(torch.bfloat16)
    rows[:, 8 * H:] *= scale
    dev = rows.cuda()
    q_out = torch.empty((n, 8 * H, D), dtype=torch.bfloat16, device="cuda")
    at, req = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    step.append(dev[:, :8 * H], dev[:, 8 * H:9 * H], dev[:, 9 * H:], at, req, q_out=q_out)
    assert int(step.status.item()) == 0
    return skv.Kv4Step(p, pool).gather()[1][0].double().cpu(), rows[:, 9 * H:].double()


@pytest.mark.parametrize("H", [1, 2, 3, 5])
def test_steps_of_nothing_beside_idle_lanes(skv, H):
    """Rows of zeros, of tiny and of ordinary steps in turn, whatever the other half of their warp holds."""
    scale = torch.ones(64, 1, 1)
    scale[1::4], scale[2::4] = 0.0, 2.0 ** -110
    got, rows = append(skv, H, 64, scale)
    c, s, z = kv4_ref.quantise(rows.numpy(), 32)
    want = torch.from_numpy(kv4_ref.values(c, s, z)).transpose(0, 1)
    step = torch.from_numpy(s).repeat_interleave(32, -1).transpose(0, 1)
    # (a code next to the border of two may fall on either side; the value is rounded to bf16)
    assert torch.all((got - want).abs() <= 2.0 ** -8 * want.abs() + 1.001 * step)
    assert torch.all(((got - want).abs() <= 2.0 ** -8 * want.abs()).double().mean((1, 2)) > 0.99)
