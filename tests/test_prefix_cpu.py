"""skv_prefix_attn without a GPU: struct layout, workspace sizes and the arguments it refuses."""

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
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


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
    body = text.split("typedef struct skv_prefix {", 1)[1].split("}", 1)[0]
    names = [d.replace("*", " ").split()[-1] for d in body.split(";") if d.strip()]
    assert names == [f for f, _ in B.CPrefix._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "skv.h"\nint main(void) {printf("%zu", '
                   "sizeof(skv_prefix));" + "".join(f'printf(" %zu", offsetof(skv_prefix, {n}));' for n in names)
                   + "return 0;}")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(B.CPrefix)] + [getattr(B.CPrefix, n).offset for n in names]


def _problem(B, **over):
    p = B.CProblem(4, 2, 8, 128, 128, 128, 8, 1000, 0, 0, 0, 16, 0, 0, 0.0, 0, FAKE)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _call(B, q=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40, problem=None, pool=None, prefix=None, lse=None,
          dev_status=None):
    p = _problem(B, **(problem or {}))
    pl = B.CPool(FAKE, FAKE, 10, None, None, 0, FAKE, 63, 0)
    px = B.CPrefix(FAKE, 500, 0)
    for obj, over in ((pl, pool), (px, prefix)):
        for k, v in (over or {}).items():
            setattr(obj, k, v)
    return B.lib().skv_prefix_attn(ctypes.byref(p), q, ctypes.byref(pl), ctypes.byref(px), out, lse, ws, ws_bytes,
                                   dev_status, None)


@pytest.mark.parametrize("over,status", [
    (dict(problem=dict(batch=0)), INVALID),
    (dict(problem=dict(n_q_heads=7)), INVALID),
    (dict(problem=dict(seq_lens=None)), INVALID),
    (dict(prefix=dict(len=-1)), INVALID),
    (dict(prefix=dict(len=1001)), INVALID),
    (dict(prefix=dict(table=None)), INVALID),
    (dict(prefix=dict(reserved=1)), INVALID),
    (dict(prefix=dict(table=FAKE + 2)), INVALID),
    (dict(q=None), INVALID),
    (dict(q=FAKE + 8), INVALID),
    (dict(out=None), INVALID),
    (dict(lse=FAKE + 2), INVALID),
    (dict(dev_status=FAKE + 2), INVALID),
    (dict(problem=dict(seq_lens=FAKE + 2)), INVALID),
    (dict(pool=dict(slot_table=FAKE + 2)), INVALID),
    (dict(ws=None), INVALID),
    (dict(ws=FAKE + 8), INVALID),
    (dict(ws_bytes=100), WORKSPACE),
    (dict(pool=dict(table_stride=62)), INVALID),
    (dict(pool=dict(gpu_k=None)), INVALID),
    (dict(pool=dict(table_heads=1)), UNSUPPORTED),
    (dict(pool=dict(gpu_v=None)), UNSUPPORTED),
    (dict(problem=dict(dtype=1)), UNSUPPORTED),
    (dict(problem=dict(d_qk=64)), UNSUPPORTED),
    (dict(problem=dict(d_v=64)), UNSUPPORTED),
    (dict(problem=dict(n_q_heads=258, n_idx_q_heads=258)), UNSUPPORTED),
])
def test_refusals(B, over, status):
    n0 = B.lib().skv_launch_count()
    assert _call(B, **over) == status
    assert B.lib().skv_launch_count() == n0


def _size(B, prefix_len, **over):
    n = ctypes.c_size_t(0)
    p = _problem(B, **over)
    st = B.lib().skv_prefix_workspace_size(ctypes.byref(p), prefix_len, ctypes.byref(n))
    return st, n.value


def test_workspace_size(B):
    st, n = _size(B, 500)
    assert st == 0 and n > 0
    assert _size(B, 1001)[0] == INVALID and _size(B, -1)[0] == INVALID
    assert _size(B, 0)[0] == 0
    assert _size(B, 1000)[1] < n  # no tails: no tail partials
    p = _problem(B)
    assert B.lib().skv_prefix_workspace_size(ctypes.byref(p), 500, None) == INVALID


def test_prefix_checks_its_table(B):
    p = B.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0, n_local=0,
                  block_size=16, seq_lens=torch.zeros(4, dtype=torch.int32))
    B.Prefix(torch.zeros(3, dtype=torch.int32), 48).check(p)
    B.Prefix(None, 0).check(p)
    for bad in (B.Prefix(None, 1), B.Prefix(torch.zeros(3, dtype=torch.int32), 49),
                B.Prefix(torch.zeros(3, dtype=torch.int64), 48), B.Prefix(torch.zeros(6, dtype=torch.int32)[::2], 48)):
        with pytest.raises(ValueError):
            bad.check(p)


def test_prefix_checks_its_length_and_device(B):
    p = B.Problem(batch=4, n_kv_heads=2, n_q_heads=8, d_qk=128, d_v=128, max_len=100, topk=0, n_sink=0, n_local=0,
                  block_size=16, seq_lens=torch.zeros(4, dtype=torch.int32))
    table = torch.zeros(7, dtype=torch.int32)
    B.Prefix(table, 100).check(p)
    for n in (-1, 101, 2 ** 32 + 5):  # the last is 5 in 32 bits
        with pytest.raises(ValueError):
            B.Prefix(table, n).check(p)
    with pytest.raises(ValueError):
        B.Prefix(table.to("meta"), 100).check(p)


def test_pairs_of_heads_and_requests_stay_in_32_bits(B):
    over = dict(batch=65535, n_kv_heads=65535, n_q_heads=65535, n_idx_q_heads=65535, max_len=16)
    assert _size(B, 0, **over)[0] == UNSUPPORTED
    assert _size(B, 0, **{**over, "batch": 1000})[0] == 0
