"""The step helpers that marshal their tensors once keep them alive, whatever becomes of the objects."""

import weakref

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def skv():
    __graft_entry__.build()
    import top_sparse_kv_gb300 as m

    return m


def _problem(skv):
    return skv.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0, n_local=0,
                       block_size=16, seq_lens=torch.zeros(4, dtype=torch.int32))


def _pool(skv):
    k, v = (torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16) for _ in range(2))
    return skv.Pool(k, v, torch.zeros((4, 7), dtype=torch.int32))


def _replace_all(objs):
    """Every tensor of the objects replaced; weak references to the ones that were there."""
    refs = []
    for o in objs:
        for name, t in list(vars(o).items()):
            if isinstance(t, torch.Tensor):
                refs.append(weakref.ref(t))
                setattr(o, name, torch.zeros(1))
    return refs


def test_token_step(skv):
    objs = [_problem(skv), skv.Rotary(torch.zeros(64), 128, k_gamma=torch.ones(128, dtype=torch.bfloat16)), _pool(skv)]
    step = skv.TokenStep(*objs)
    refs = _replace_all(objs)
    assert len(refs) == 6 and all(r() is not None for r in refs)
    del step, objs
    assert all(r() is None for r in refs)


def test_prefix_step(skv):
    objs = [_problem(skv), _pool(skv), skv.Prefix(torch.zeros(3, dtype=torch.int32), 48)]
    step = skv.PrefixStep(*objs)
    refs = _replace_all(objs)
    assert len(refs) == 5 and all(r() is not None for r in refs)
    del step, objs
    assert all(r() is None for r in refs)
