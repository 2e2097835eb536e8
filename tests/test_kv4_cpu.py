"""The cache in 4 bits and the block tables without a GPU: struct layout, the arguments they refuse."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import __graft_entry__
import kv4_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned, never-dereferenced address: validation rejects before use


@pytest.fixture(scope="module")
def B():
    __graft_entry__.build()
    from top_sparse_kv_gb300 import binding

    return binding


def test_struct_layout(B, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    text = re.sub(r"/\*.*?\*/", " ", open(os.path.join(ROOT, "include", "skv.h")).read(), flags=re.S)
    body = text.split("typedef struct skv_tables {", 1)[1].split("}", 1)[0]
    fields = [f for f, _ in B.CTables._fields_]
    assert [d.replace("*", " ").split()[-1] for d in body.split(";") if d.strip()] == fields
    src = tmp_path / "l.c"
    src.write_text("\n".join(["#include <stdio.h>", "#include <stddef.h>", '#include "skv.h"', "int main(void) {",
                              'printf("%zu\\n", sizeof(skv_tables));']
                             + [f'printf("%zu\\n", offsetof(skv_tables, {f}));' for f in fields] + ["return 0;", "}"]))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(B.CTables)] + [getattr(B.CTables, f).offset for f in fields]


def _tables(B, **over):
    t = B.CTables(4, 1000, 16, 0, 63, 100, FAKE, FAKE, FAKE, FAKE)
    for k, v in over.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), 1), (dict(max_len=-1), 1), (dict(block_size=0), 1), (dict(base=-1), 1), (dict(base=1001), 1),
    (dict(table_stride=62), 1), (dict(n_blocks=-1), 1), (dict(slot_table=None), 1), (dict(seq_lens=None), 1),
    (dict(free_blocks=None), 1), (dict(state=None), 1), (dict(state=FAKE + 2), 1), (dict(seq_lens=FAKE + 1), 1),
    (dict(batch=4097), 2),
])
def test_tables_refusals(B, over, status):
    t = _tables(B, **over)
    assert B.lib().skv_update_tables(ctypes.byref(t), FAKE, 4, FAKE, FAKE, None, None, None) == status


@pytest.mark.parametrize("args", [
    (None, 4, FAKE, FAKE, None, None), (FAKE, -1, FAKE, FAKE, None, None), (FAKE, 4, None, FAKE, None, None),
    (FAKE, 4, FAKE, None, None, None), (FAKE, 4, FAKE + 4, FAKE, None, None), (FAKE, 4, FAKE, FAKE, FAKE + 8, None),
    (FAKE, 4, FAKE, FAKE, None, FAKE + 2), (FAKE + 2, 4, FAKE, FAKE, None, None),
])
def test_tables_call_refusals(B, args):
    t = _tables(B)
    assert B.lib().skv_update_tables(ctypes.byref(t), *args, None) == 1
    assert B.lib().skv_update_tables(None, *args, None) == 1


def _problem(B, **over):
    p = B.CProblem(4, 2, 8, 128, 128, 128, 8, 1000, 100, 4, 64, 16, 0, 0, 0.0, 0, FAKE)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _pool(B, **over):
    p = B.CPool(FAKE, FAKE, 10, None, None, 0, FAKE, 63, 0)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _calls(B, p, pool, group=32, q=FAKE, ws=FAKE, ws_bytes=1 << 40):
    """The status of each call."""
    L, P, PL = B.lib(), ctypes.byref(p), ctypes.byref(pool)
    rot, tok = B.CRotary(0, 128, 0, 0, 1e-6, FAKE, FAKE, FAKE), B.CTokens(4, 0, FAKE, FAKE, FAKE, 1024, 256, 256, None, None)
    return dict(append=L.skv_append_kv4(P, ctypes.byref(rot), ctypes.byref(tok), PL, group, q, None, None),
                gather=L.skv_gather_kv4(P, PL, group, FAKE, q, FAKE, None, None),
                score=L.skv_score_kv4(P, q, PL, group, FAKE, None, None),
                attn=L.skv_attn_kv4(P, q, PL, group, FAKE, FAKE, FAKE, ws, ws_bytes, None, None),
                step=L.skv_decode_step_kv4(P, q, None, PL, group, FAKE, FAKE, FAKE, FAKE, ws, ws_bytes, None, None))


@pytest.mark.parametrize("problem,pool,kw,status", [
    (dict(batch=0), {}, {}, 1), (dict(seq_lens=None), {}, {}, 1), (dict(seq_lens=FAKE + 2), {}, {}, 1),
    ({}, {}, dict(group=16), 1), ({}, {}, dict(group=0), 1), ({}, {}, dict(group=256), 1),
    ({}, dict(gpu_k=None), {}, 1), ({}, dict(gpu_k=FAKE + 8), {}, 1), ({}, dict(slot_table=None), {}, 1),
    ({}, dict(slot_table=FAKE + 2), {}, 1), ({}, dict(table_stride=62), {}, 1), ({}, dict(table_heads=2), {}, 1),
    ({}, dict(host_k=FAKE), {}, 1), ({}, {}, dict(q=FAKE + 8), 1),
    (dict(block_size=8), {}, {}, 1), (dict(block_size=24), {}, {}, 2), (dict(block_size=17), {}, {}, 2),
    (dict(d_qk=64, d_v=64), {}, {}, 2), (dict(n_q_heads=34), {}, {}, 2), (dict(max_len=(1 << 30) + 1), dict(table_stride=1 << 27), {}, 2),
    ({}, dict(gpu_v=None), {}, 2), (dict(topk=1 << 30, n_local=1 << 20), {}, {}, 2),
])
def test_kv4_refusals(B, problem, pool, kw, status):
    got = _calls(B, _problem(B, **problem), _pool(B, **pool), **kw)
    if problem.get("n_q_heads") == 34:
        got.pop("append")  # (34 heads do not fit its strides: refused for that)
    assert set(got.values()) == {status}, got


def test_kv4_call_refusals(B):
    p, pl, L = _problem(B), _pool(B), B.lib()
    P, PL = ctypes.byref(p), ctypes.byref(pl)
    n = ctypes.c_size_t(0)
    assert L.skv_kv4_workspace_size(P, ctypes.byref(n)) == 0 and n.value > 0
    assert L.skv_kv4_workspace_size(P, None) == 1 and L.skv_kv4_workspace_size(None, ctypes.byref(n)) == 1
    assert L.skv_attn_kv4(P, FAKE, PL, 32, FAKE, FAKE, FAKE, FAKE, 100, None, None) == 4
    assert L.skv_attn_kv4(P, FAKE, PL, 32, FAKE, FAKE, FAKE, None, 1 << 40, None, None) == 1
    assert L.skv_attn_kv4(P, FAKE, PL, 32, FAKE, None, FAKE, FAKE, 1 << 40, None, None) == 1
    assert L.skv_attn_kv4(P, FAKE, PL, 32, FAKE + 2, FAKE, FAKE, FAKE, 1 << 40, None, None) == 1
    assert L.skv_attn_kv4(P, FAKE, PL, 32, FAKE, FAKE, FAKE + 2, FAKE, 1 << 40, None, None) == 1
    assert L.skv_decode_step_kv4(P, FAKE, None, PL, 32, None, FAKE, FAKE, FAKE, FAKE, 1 << 40, None, None) == 1
    assert L.skv_decode_step_kv4(P, FAKE, None, PL, 32, FAKE, FAKE, FAKE, FAKE, FAKE, 100, None, None) == 4
    assert L.skv_gather_kv4(P, PL, 32, None, FAKE, FAKE, None, None) == 1  # a selection is missing
    assert L.skv_gather_kv4(P, PL, 32, FAKE, None, None, None, None) == 1
    assert L.skv_score_kv4(P, FAKE, PL, 32, FAKE + 4, None, None) == 1
    f32 = _problem(B, dtype=1)
    got = _calls(B, f32, pl)
    assert got["score"] == got["attn"] == got["step"] == 2
    # no tokens: nothing is enqueued
    rot, tok = B.CRotary(0, 128, 0, 0, 1e-6, FAKE, FAKE, FAKE), B.CTokens(0, 0, None, None, None, 0, 0, 0, None, None)
    assert L.skv_append_kv4(P, ctypes.byref(rot), ctypes.byref(tok), PL, 32, None, None, None) == 0
    none = _problem(B, topk=0, n_sink=0, n_local=0)
    assert L.skv_gather_kv4(ctypes.byref(none), PL, 32, None, FAKE, FAKE, None, None) == 0


def _py(B, **kw):
    lens = torch.zeros(4, dtype=torch.int32)
    p = B.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=5, n_sink=1, n_local=2,
                  block_size=16, seq_lens=lens)
    pool = B.Kv4Pool.empty(10, 2, 16, torch.zeros((4, 7), dtype=torch.int32), **kw)
    return p, pool


def test_python_refusals(B):
    import top_sparse_kv_gb300 as skv

    p, pool = _py(B)
    assert pool.gpu_k.shape == (10, 2, 1, 1280)
    for wrong in (dict(gpu_k=pool.gpu_k.float()), dict(gpu_v=pool.gpu_v[:9]), dict(gpu_v=None), dict(group=16),
                  dict(group=64), dict(host_k=pool.gpu_k), dict(slot_table=pool.slot_table.long()),
                  dict(slot_table=pool.slot_table[:3])):
        bad = B.Kv4Pool(**{**vars(pool), **wrong})
        with pytest.raises(ValueError):
            skv.Kv4Step(p, bad)
    plain = B.Pool(torch.zeros((10, 2, 16, 128), dtype=torch.bfloat16), torch.zeros((10, 2, 16, 128), dtype=torch.bfloat16),
                   pool.slot_table)
    with pytest.raises(ValueError):
        skv.Kv4Step(p, plain)
    # the calls of other pools do not take one in 4 bits
    idx = torch.zeros((4, 2, 5), dtype=torch.int32)
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        skv.skv_sparse_attn(p, q, pool, idx, q, None, q)
    with pytest.raises(ValueError):
        skv.skv_score(p, q, skv.IndexSrc(), pool, torch.zeros((4, 2, 100)))
    with pytest.raises(ValueError):
        skv.PrefixStep(p, pool, skv.Prefix(None, 0))
    with pytest.raises(ValueError):
        skv.SlotCache.from_table(p, pool, 4)
    step = skv.Kv4Step(p, pool)
    for bad in (q.float(), q[:3], torch.zeros((4, 128, 8), dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(ValueError):
            step.attend_all(bad)
    with pytest.raises(ValueError):
        step.attend(q, idx.long())
    with pytest.raises(ValueError):
        step.gather(idx[:, :1])
    with pytest.raises(ValueError):
        step.score(q, torch.zeros((4, 2, 99)))


def test_python_tables_refusals(B):
    import top_sparse_kv_gb300 as skv

    p, pool = _py(B)
    free = torch.arange(10, dtype=torch.int32)
    for args, kw in (((pool.slot_table[:3], free), {}), ((pool.slot_table, free.long()), {}),
                     ((pool.slot_table.view(-1), free), {}), ((pool.slot_table, free), dict(n_free=11)),
                     ((pool.slot_table, free), dict(n_free=-1))):
        with pytest.raises(ValueError):
            skv.BlockTables(p, *args, **kw)
    t = skv.BlockTables(p, pool.slot_table, free, n_free=7)
    assert t.n_free.tolist() == [7]
    with pytest.raises(ValueError):
        t.update(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        t.update(torch.zeros(3, dtype=torch.int32))
    rows = (torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        t.update(torch.zeros(4, dtype=torch.int32), 4, out=rows)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_reference_cells(group):
    """The reference's own two ways agree, and a row comes back within half a step (and what the ends lose)."""
    rng = np.random.default_rng(group)
    cache = kv4_ref.Cache(3, 2, 32, group, rng)
    x = rng.standard_normal((40, 128)) * np.exp(rng.standard_normal((40, 1)))
    at = rng.permutation(3 * 2 * 32)[:40]
    e, h, t = at // 64, at // 32 % 2, at % 32
    cache.put(e, h, t, x)
    c, s, z = cache.raw(e, h, t)
    rep = lambda a: np.repeat(a, group, -1)  # noqa: E731
    assert np.all(np.abs(kv4_ref.values(c, s, z) - x) <= rep(s) * (0.5 + 2.0 ** -5) + 2.0 ** -8 * np.abs(rep(z)))
