"""skv_append_kv_cached without a GPU: the arguments it refuses."""

import ctypes

import pytest
import torch

import __graft_entry__

FAKE = 1 << 20  # an aligned, never-dereferenced address: validation rejects before use
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def B():
    __graft_entry__.build()
    from top_sparse_kv_gb300 import binding

    return binding


def _call(B, latent=False, problem=None, tokens=None, pool=None, q_out=FAKE):
    if latent:
        p = B.CProblem(4, 1, 8, 128, 576, 512, 8, 1000, 0, 0, 0, 1, 0, 0, 0.0, 0, FAKE)
        pl = B.CPool(FAKE, None, 10, FAKE, None, 4000, FAKE, 1000, 0)
    else:
        p = B.CProblem(4, 2, 8, 128, 128, 128, 8, 1000, 0, 0, 0, 16, 0, 0, 0.0, 0, FAKE)
        pl = B.CPool(FAKE, FAKE, 10, FAKE, FAKE, 252, FAKE, 63, 1)
    t = B.CTokens(0, 0, FAKE, FAKE, FAKE, 8 * 576, 576, 512, None, None)
    r = B.CRotary(0, 0, 0, 0, 1e-6, None, None, None)
    for obj, over in ((p, problem), (t, tokens), (pl, pool)):
        for k, v in (over or {}).items():
            setattr(obj, k, v)
    n0 = B.lib().skv_launch_count()
    st = B.lib().skv_append_kv_cached(ctypes.byref(p), ctypes.byref(r), ctypes.byref(t), ctypes.byref(pl), q_out, None,
                                      None)
    assert B.lib().skv_launch_count() == n0
    return st


def test_both_caches_are_taken(B):
    assert _call(B) == 0 and _call(B, latent=True) == 0


@pytest.mark.parametrize("latent,over,status", [
    (False, dict(pool=dict(n_host_blocks=251)), UNSUPPORTED),   # a block without its host block
    (False, dict(pool=dict(host_k=None, host_v=None)), INVALID),
    (False, dict(pool=dict(host_v=None)), INVALID),
    (False, dict(pool=dict(host_k=FAKE + 8)), INVALID),
    (False, dict(pool=dict(table_heads=0)), UNSUPPORTED),       # K and V pools: per-head tables alone
    (False, dict(pool=dict(n_gpu_blocks=0)), UNSUPPORTED),
    (False, dict(problem=dict(batch=1024)), UNSUPPORTED),       # more units than the cache has
    (False, dict(tokens=dict(reserved=1)), INVALID),
    (True, dict(pool=dict(n_host_blocks=3999)), UNSUPPORTED),
    (True, dict(pool=dict(host_k=None)), INVALID),
    (True, dict(problem=dict(block_size=16)), UNSUPPORTED),
    (True, dict(problem=dict(batch=65)), UNSUPPORTED),
    (True, dict(pool=dict(slot_table=None)), INVALID),
])
def test_refusals(B, latent, over, status):
    assert _call(B, latent, **over) == status


def test_a_cache_that_cannot_be_made_leaves_the_pool_alone(B):
    p = B.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0, n_local=0,
                  block_size=1, seq_lens=torch.zeros(4, dtype=torch.int32))
    k, v = (torch.zeros((28, 2, 1, 128), dtype=torch.bfloat16) for _ in range(2))
    pool = B.Pool(k, v, torch.full((4, 100), -1, dtype=torch.int32))  # one table for all heads: no cache of it
    with pytest.raises(B.SkvError):
        B.SlotCache.from_table(p, pool, 4)
    assert not pool.cached
