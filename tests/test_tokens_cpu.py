"""skv_qk_norm_rope / skv_append_kv without a GPU: struct layouts, and the arguments they refuse."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned, never-dereferenced address: validation rejects before use


@pytest.fixture(scope="module")
def B():
    __graft_entry__.build()
    from top_sparse_kv_gb300 import binding

    return binding


def test_struct_layouts(B, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    structs = {"skv_rotary": B.CRotary, "skv_tokens": B.CTokens}
    text = re.sub(r"/\*.*?\*/", " ", open(os.path.join(ROOT, "include", "skv.h")).read(), flags=re.S)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "skv.h"', "int main(void) {"]
    for cname, cls in structs.items():
        body = text.split(f"typedef struct {cname} {{", 1)[1].split("}", 1)[0]
        assert [d.replace("*", " ").split()[-1] for d in body.split(";") if d.strip()] == [f for f, _ in cls._fields_]
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        lines += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    want = []
    for cls in structs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def _args(B, problem=None, rotary=None, tokens=None, pool=None):
    p = B.CProblem(4, 2, 8, 128, 128, 128, 8, 1000, 0, 0, 0, 16, 0, 0, 0.0, 0, FAKE)
    r = B.CRotary(0, 128, 0, 0, 1e-6, FAKE, FAKE, FAKE)
    t = B.CTokens(4, 0, FAKE, FAKE, FAKE, 1024, 256, 256, None, None)
    pl = B.CPool(FAKE, FAKE, 10, None, None, 0, FAKE, 63, 0)
    for obj, over in ((p, problem), (r, rotary), (t, tokens), (pl, pool)):
        for k, v in (over or {}).items():
            setattr(obj, k, v)
    return p, r, t, pl


def _append(B, q_out=FAKE, dev_status=None, **over):
    p, r, t, pl = _args(B, **over)
    return B.lib().skv_append_kv(ctypes.byref(p), ctypes.byref(r), ctypes.byref(t), ctypes.byref(pl), q_out, dev_status,
                                 None)


def _norm(B, q_out=FAKE, k_out=FAKE, dev_status=None, **over):
    p, r, t, _ = _args(B, **over)
    return B.lib().skv_qk_norm_rope(ctypes.byref(p), ctypes.byref(r), ctypes.byref(t), q_out, k_out, dev_status, None)


INVALID, UNSUPPORTED = 1, 2

BOTH = [
    (dict(problem=dict(batch=0)), INVALID),
    (dict(problem=dict(seq_lens=None)), INVALID),
    (dict(tokens=dict(n_tokens=-1)), INVALID),
    (dict(tokens=dict(reserved=1)), INVALID),
    (dict(tokens=dict(q=FAKE + 8)), INVALID),
    (dict(tokens=dict(k=FAKE + 2)), INVALID),
    (dict(tokens=dict(q_stride=1020)), INVALID),   # less than a row
    (dict(tokens=dict(q_stride=1028)), INVALID),   # rows off the 16-byte grid
    (dict(tokens=dict(k_stride=-256)), INVALID),
    (dict(rotary=dict(style=2)), INVALID),
    (dict(rotary=dict(eps=-1.0)), INVALID),
    (dict(rotary=dict(eps=float("nan"))), INVALID),
    (dict(rotary=dict(rot_start=8)), INVALID),     # past the row's end
    (dict(rotary=dict(rot_dim=136)), INVALID),
    (dict(rotary=dict(norm_dim=136)), INVALID),
    (dict(rotary=dict(inv_freq=None)), INVALID),
    (dict(rotary=dict(q_gamma=FAKE + 4)), INVALID),
    (dict(rotary=dict(inv_freq=FAKE + 2)), INVALID),
    (dict(tokens=dict(positions=FAKE + 2)), INVALID),
    (dict(tokens=dict(requests=FAKE + 2)), INVALID),
    (dict(problem=dict(seq_lens=FAKE + 2)), INVALID),
    (dict(dev_status=FAKE + 2), INVALID),
    (dict(rotary=dict(rot_dim=120)), UNSUPPORTED),  # halves that split a vector
    (dict(rotary=dict(rot_dim=116, style=1)), UNSUPPORTED),
    (dict(rotary=dict(rot_start=4, rot_dim=64)), UNSUPPORTED),
    (dict(rotary=dict(norm_dim=100)), UNSUPPORTED),
    (dict(tokens=dict(n_tokens=5)), INVALID),       # more tokens than requests, no request ids
]


@pytest.mark.parametrize("over,status", BOTH)
def test_both_refuse(B, over, status):
    n0 = B.lib().skv_launch_count()
    assert _append(B, **over) == status
    assert _norm(B, **over) == status
    assert B.lib().skv_launch_count() == n0


@pytest.mark.parametrize("over,status", [
    (dict(q_out=None), INVALID),
    (dict(tokens=dict(k=None)), INVALID),
    (dict(tokens=dict(v=None)), INVALID),
    (dict(tokens=dict(v=FAKE + 8)), INVALID),
    (dict(tokens=dict(v_stride=100)), INVALID),
    (dict(pool=dict(gpu_k=None)), INVALID),
    (dict(pool=dict(table_stride=62)), INVALID),
    (dict(pool=dict(slot_table=FAKE + 2)), INVALID),
    (dict(pool=dict(gpu_v=None)), INVALID),          # the latent layout has one KV head
    (dict(problem=dict(d_v=1032)), UNSUPPORTED),
])
def test_append_refuses(B, over, status):
    if "d_v" in over.get("problem", {}):
        over = dict(over, tokens=dict(v_stride=4096))
    assert _append(B, **over) == status


def test_norm_refuses_missing_outputs(B):
    assert _norm(B, k_out=None) == INVALID
    assert _norm(B, q_out=None) == INVALID
    assert _norm(B, q_out=None, k_out=None, tokens=dict(q=None, k=None)) == INVALID


def test_no_tokens_is_a_call_that_does_nothing(B):
    n0 = B.lib().skv_launch_count()
    assert _append(B, tokens=dict(n_tokens=0)) == 0
    assert _norm(B, tokens=dict(n_tokens=0)) == 0
    assert B.lib().skv_launch_count() == n0


def test_binding_checks_types_and_shapes(B):
    lens = torch.zeros(4, dtype=torch.int32)
    p = B.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0, n_local=0,
                  block_size=16, seq_lens=lens)
    q, k, v = (torch.zeros((4, h, 128), dtype=torch.bfloat16) for h in (8, 2, 2))
    assert B.c_tokens(p, q, k, v, lens, None).q_stride == 1024
    fused = torch.zeros((4, 12 * 128), dtype=torch.bfloat16)
    assert B.c_tokens(p, fused[:, :1024].view(4, 8, 128), k, v, None, None).q_stride == 12 * 128
    for bad in ((q.float(), k, v), (q[:3], k, v), (q, k[:, :1], v), (q, k, v[..., :64]),
                (q.transpose(0, 1).contiguous().transpose(0, 1), k, v)):
        with pytest.raises(ValueError):
            B.c_tokens(p, *bad, None, None)
    with pytest.raises(ValueError):
        B.c_tokens(p, q, k, v, lens.long(), None)
    with pytest.raises(ValueError):
        B.c_tokens(p, q, k, v, lens[:3], None)
    for bad in (dict(inv_freq=torch.zeros(64, dtype=torch.float64)), dict(inv_freq=torch.zeros(32)),
                dict(inv_freq=None), dict(inv_freq=torch.zeros(64), q_gamma=torch.zeros(128)),
                dict(inv_freq=torch.zeros(64), k_gamma=torch.zeros(64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            B.Rotary(rot_dim=128, **bad).check(p)


def test_no_rows_may_be_null_pointers(B):
    """What an empty tensor's address is."""
    n0 = B.lib().skv_launch_count()
    none = dict(n_tokens=0, q=None, k=None, v=None)
    assert _append(B, tokens=none, q_out=None) == 0
    assert _norm(B, tokens=none, q_out=None, k_out=None) == 0
    assert B.lib().skv_launch_count() == n0


def _problem(B, **over):
    return B.Problem(**{**dict(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0,
                               n_local=0, block_size=16, seq_lens=torch.zeros(4, dtype=torch.int32)), **over})


def _pool(B, n=5, dtype=torch.bfloat16, **over):
    kv = [torch.zeros((n, 2, 16, 128), dtype=dtype) for _ in range(2)]
    return B.Pool(**{**dict(gpu_k=kv[0], gpu_v=kv[1], slot_table=torch.zeros((4, 7), dtype=torch.int32)), **over})


def test_outputs_go_with_their_inputs(B):
    fused = torch.zeros((4, 12 * 128), dtype=torch.bfloat16)
    q = fused[:, :1024].view(4, 8, 128)
    bf = torch.bfloat16
    B._out_rows("q_out", q, q, 8, 128, bf)
    B._out_rows("q_out", torch.zeros((4, 8, 128), dtype=bf), q, 8, 128, bf)
    # packed rows from the input's own address on would be taken for the input in place
    with pytest.raises(ValueError):
        B._out_rows("q_out", fused.view(-1)[:4096].view(4, 8, 128), q, 8, 128, bf)
    with pytest.raises(ValueError):
        B._out_rows("q_out", torch.zeros((4, 12 * 128), dtype=bf)[:, :1024].view(4, 8, 128), q, 8, 128, bf)
    with pytest.raises(ValueError):
        B._out_rows("k_out", q, None, 8, 128, bf)


def test_tensors_of_another_device(B):
    """Nothing of one device's reaches a kernel of another's ("meta" stands for the other here)."""
    p, rot = _problem(B), B.Rotary(torch.zeros(64), 128)
    q, k, v = (torch.zeros((4, h, 128), dtype=torch.bfloat16) for h in (8, 2, 2))
    ids = torch.zeros(4, dtype=torch.int32)
    for i in range(5):
        args = [q, k, v, ids, ids]
        args[i] = args[i].to("meta")
        with pytest.raises(ValueError):
            B.c_tokens(p, *args)
    with pytest.raises(ValueError):
        B.Rotary(torch.zeros(64, device="meta"), 128).check(p)
    with pytest.raises(ValueError):
        B._out_rows("q_out", q.to("meta"), q, 8, 128, torch.bfloat16)
    for name in ("gpu_k", "gpu_v", "slot_table"):
        with pytest.raises(ValueError):
            B.check_pool(p, _pool(B, **{name: getattr(_pool(B), name).to("meta")}))
    import top_sparse_kv_gb300 as skv

    with pytest.raises(ValueError):  # and the CPU's reach no kernel at all
        skv.TokenStep(p, rot).norm_rope(q, k)


def test_pool_is_the_problems(B):
    p = _problem(B)
    B.check_pool(p, _pool(B))
    bad = [_pool(B, dtype=torch.float32), _pool(B, gpu_k=torch.zeros((5, 2, 8, 128), dtype=torch.bfloat16)),
           _pool(B, slot_table=torch.zeros((3, 7), dtype=torch.int32)),
           _pool(B, slot_table=torch.zeros((4, 7), dtype=torch.int64)),
           _pool(B, slot_table=torch.zeros((4, 14), dtype=torch.int32)[:, ::2]),
           _pool(B, host_k=torch.zeros((5, 1, 16, 128), dtype=torch.bfloat16))]
    for pool in bad:
        with pytest.raises(ValueError):
            B.check_pool(p, pool)
    with pytest.raises(ValueError):
        B.check_pool(_problem(B, seq_lens=torch.zeros(3, dtype=torch.int32)), _pool(B))
