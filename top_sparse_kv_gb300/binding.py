"""ctypes binding of libskv.so: the C ABI's names, argument marshalling only.

Every function takes torch tensors (device memory, or pinned host memory for
host pools), passes their raw pointers to the C entry point of the same name
and raises SkvError on a non-OK status.  No arithmetic of the step happens
here; if the library is missing the import fails loudly -- there is no
fallback path.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libskv.so")

SKV_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "CUDA error",
                4: "workspace too small", 5: "device fault", 6: "timeout"}
SKV_DEV_BAD_SLOT, SKV_DEV_BAD_INDEX, SKV_DEV_BAD_LENGTH, SKV_DEV_TIMEOUT = 1, 2, 4, 8
SKV_DEV_NO_BLOCK = 16
SKV_DTYPE_BF16, SKV_DTYPE_F32 = 0, 1
SKV_AGG_MEAN = 0
SKV_AGG_MAX = 1
SKV_AGG_HEAD = 2  # every query head selects its own top-k
SKV_INDEX_PAGED, SKV_INDEX_CONTIG = 0, 1
SKV_ROPE_HALF, SKV_ROPE_PAIR = 0, 1


class SkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} (status {status})")
        self.status = status


class CProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "n_kv_heads", "n_q_heads", "d_qk", "d_v", "d_idx", "n_idx_q_heads", "max_len",
        "topk", "n_sink", "n_local", "block_size", "dtype", "group_agg")] + [
        ("sm_scale", ctypes.c_float), ("n_splits", ctypes.c_int32), ("seq_lens", ctypes.c_void_p)]


class CPool(ctypes.Structure):
    _fields_ = [("gpu_k", ctypes.c_void_p), ("gpu_v", ctypes.c_void_p), ("n_gpu_blocks", ctypes.c_int64),
                ("host_k", ctypes.c_void_p), ("host_v", ctypes.c_void_p), ("n_host_blocks", ctypes.c_int64),
                ("slot_table", ctypes.c_void_p), ("table_stride", ctypes.c_int32), ("table_heads", ctypes.c_int32)]


class CIndex(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("keys", ctypes.c_void_p)]


class CSlotCache(ctypes.Structure):
    _fields_ = [("owner", ctypes.c_void_p), ("prio", ctypes.c_void_p), ("step", ctypes.c_void_p),
                ("budget", ctypes.c_int32), ("stats", ctypes.c_void_p)]


class CParis(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("beta_pm", ctypes.c_int32), ("rho_pm", ctypes.c_int32),
                ("signs", ctypes.c_void_p)]


class CParisIndex(ctypes.Structure):
    _fields_ = [("cent", ctypes.c_void_p), ("rec", ctypes.c_void_p), ("hist", ctypes.c_void_p)]


class CRotary(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rot_start", "rot_dim", "style", "norm_dim")] + [
        ("eps", ctypes.c_float), ("inv_freq", ctypes.c_void_p), ("q_gamma", ctypes.c_void_p),
        ("k_gamma", ctypes.c_void_p)]


class CTokens(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("requests", ctypes.c_void_p)]


class CPrefix(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("len", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CTables(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "max_len", "block_size", "base", "table_stride", "n_blocks")] + [
        (n, ctypes.c_void_p) for n in ("slot_table", "seq_lens", "free_blocks", "state")]


class CPrefetch(ctypes.Structure):
    _fields_ = [("tau_ema", ctypes.c_void_p), ("epoch", ctypes.c_void_p), ("map", ctypes.c_void_p),
                ("staging", ctypes.c_void_p), ("count", ctypes.c_void_p), ("stats", ctypes.c_void_p),
                ("cap", ctypes.c_int32), ("alpha", ctypes.c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libskv.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                          "or python -m top_sparse_kv_gb300.build_lib")
    lib = ctypes.CDLL(LIB_PATH)
    P, VP, SZ = ctypes.POINTER(CProblem), ctypes.c_void_p, ctypes.c_size_t
    sig = {
        "skv_workspace_size": [P, ctypes.POINTER(ctypes.c_size_t)],
        "skv_score": [P, VP, ctypes.POINTER(CIndex), ctypes.POINTER(CPool), VP, VP, VP],
        "skv_topk": [P, VP, VP, VP, SZ, VP, VP],
        "skv_gather": [P, ctypes.POINTER(CPool), VP, VP, VP, VP, VP],
        "skv_sparse_attn": [P, VP, ctypes.POINTER(CPool), VP, VP, VP, VP, SZ, VP, VP],
        "skv_decode_step": [P, VP, VP, ctypes.POINTER(CIndex), ctypes.POINTER(CPool), VP, VP, VP, VP, VP, SZ,
                            VP, VP],
        "skv_decode_step_prefetch": [P, VP, VP, ctypes.POINTER(CIndex), ctypes.POINTER(CPool), VP, VP, VP, VP,
                                     VP, SZ, ctypes.POINTER(CPrefetch), VP, VP],
        "skv_cache_workspace_size": [P, ctypes.POINTER(CPool), ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
        "skv_decode_step_cached": [P, VP, VP, ctypes.POINTER(CIndex), ctypes.POINTER(CPool), VP, VP, VP, VP, VP,
                                   SZ, ctypes.POINTER(CSlotCache), VP, SZ, VP, VP],
        "skv_cache_prepare": [],
        "skv_cache_update": [P, ctypes.POINTER(CPool), VP, VP, SZ, ctypes.POINTER(CSlotCache), VP, SZ, VP, VP],
        "skv_paris_quantizer": [ctypes.c_int32, VP, VP],
        "skv_paris_encode": [P, ctypes.POINTER(CParis), ctypes.POINTER(CIndex), ctypes.POINTER(CPool),
                             ctypes.POINTER(CParisIndex), VP, VP],
        "skv_paris_workspace_size": [P, ctypes.POINTER(CParis), ctypes.POINTER(ctypes.c_size_t)],
        "skv_paris_workspace_offsets": [P, ctypes.POINTER(CParis), VP],
        "skv_paris_select": [P, ctypes.POINTER(CParis), VP, ctypes.POINTER(CIndex), ctypes.POINTER(CParisIndex),
                             ctypes.POINTER(CPool), VP, VP, SZ, VP, VP],
        "skv_paris_decode_step": [P, ctypes.POINTER(CParis), VP, VP, ctypes.POINTER(CIndex),
                                  ctypes.POINTER(CParisIndex), ctypes.POINTER(CPool), VP, VP, VP, VP, SZ, VP, VP],
        "skv_qk_norm_rope": [P, ctypes.POINTER(CRotary), ctypes.POINTER(CTokens), VP, VP, VP, VP],
        "skv_append_kv": [P, ctypes.POINTER(CRotary), ctypes.POINTER(CTokens), ctypes.POINTER(CPool), VP, VP, VP],
        "skv_append_kv_cached": [P, ctypes.POINTER(CRotary), ctypes.POINTER(CTokens), ctypes.POINTER(CPool), VP, VP,
                                 VP],
        "skv_prefix_workspace_size": [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
        "skv_prefix_attn": [P, VP, ctypes.POINTER(CPool), ctypes.POINTER(CPrefix), VP, VP, VP, SZ, VP, VP],
        "skv_update_tables": [ctypes.POINTER(CTables), VP, ctypes.c_int32, VP, VP, VP, VP, VP],
        "skv_append_kv4": [P, ctypes.POINTER(CRotary), ctypes.POINTER(CTokens), ctypes.POINTER(CPool),
                           ctypes.c_int32, VP, VP, VP],
        "skv_gather_kv4": [P, ctypes.POINTER(CPool), ctypes.c_int32, VP, VP, VP, VP, VP],
        "skv_score_kv4": [P, VP, ctypes.POINTER(CPool), ctypes.c_int32, VP, VP, VP],
        "skv_kv4_workspace_size": [P, ctypes.POINTER(ctypes.c_size_t)],
        "skv_attn_kv4": [P, VP, ctypes.POINTER(CPool), ctypes.c_int32, VP, VP, VP, VP, SZ, VP, VP],
        "skv_decode_step_kv4": [P, VP, VP, ctypes.POINTER(CPool), ctypes.c_int32, VP, VP, VP, VP, VP, SZ, VP, VP],
        "skv_block_workspace_size": [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_int32)],
        "skv_block_summaries": [P, ctypes.POINTER(CPool), VP, VP, VP],
        "skv_block_select": [P, ctypes.c_int32, VP, VP, VP, VP, VP, SZ, VP, VP],
        "skv_block_decode_step": [P, ctypes.c_int32, VP, VP, ctypes.POINTER(CPool), VP, VP, VP, VP, VP, SZ, VP,
                                  VP],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int32
    lib.skv_status_string.argtypes = [ctypes.c_int32]
    lib.skv_status_string.restype = ctypes.c_char_p
    lib.skv_launch_count.argtypes = []
    lib.skv_launch_count.restype = ctypes.c_uint64
    lib.skv_check_wait_timeout.argtypes = [ctypes.c_int64, ctypes.c_int32, VP, VP]
    lib.skv_check_wait_timeout.restype = ctypes.c_int32
    return lib


_lib = None


def lib():
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libskv must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def raw_stream(device: int, stream=None) -> int:
    """The cudaStream_t of `stream`, or of the current stream, without building a Stream object
    (torch.cuda.current_stream() costs more than a small kernel's launch).  `device`: index of
    the GPU that holds the call's tensors, which must be the current one and the stream's."""
    if device < 0 or torch._C._cuda_getDevice() != device:
        raise ValueError("the tensors must be on the current GPU")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError("the stream belongs to another GPU")
    return stream.cuda_stream


def same_device(p: "Problem", **tensors) -> int:
    """The index of the problem's device (-1: the CPU), which has to hold the tensors too."""
    for name, t in tensors.items():
        if t is not None and t.device != p.seq_lens.device:
            raise ValueError(f"{name}: on {t.device}, seq_lens on {p.seq_lens.device}")
    return p.seq_lens.get_device()


def check_lens(p: "Problem") -> None:
    t = p.seq_lens
    if t.dtype != torch.int32 or t.numel() < p.batch or not t.is_contiguous():
        raise ValueError(f"seq_lens: contiguous int32 [{p.batch}] expected")


def check_pool(p: "Problem", pool: "Pool") -> None:
    """The pool's types, sizes and devices, which the C side cannot see."""
    same_device(p, gpu_k=pool.gpu_k, gpu_v=pool.gpu_v, slot_table=pool.slot_table)
    heads = 1 if pool.table_heads else p.n_kv_heads
    if isinstance(pool, Kv4Pool):
        pool.check(p)
        sides = ()
    else:
        sides = (("gpu_k", p.d_qk), ("gpu_v", p.d_v), ("host_k", p.d_qk), ("host_v", p.d_v))
    for name, d in sides:
        t = getattr(pool, name)
        if t is None:
            continue
        rows = t.shape[0] * (p.n_kv_heads if name.startswith("host") else heads) * p.block_size
        if t.dtype != element_type(p) or t.numel() != rows * d or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous {element_type(p)} blocks of {p.block_size} rows of {d} expected")
    if pool.slot_table.dtype != torch.int32 or not pool.slot_table.is_contiguous() \
            or pool.slot_table.shape[0] < p.batch:
        raise ValueError(f"slot_table: contiguous int32, a row for each of {p.batch} requests")
    check_lens(p)


def check_pool4(p: "Problem", pool: "Kv4Pool") -> None:
    if not isinstance(pool, Kv4Pool):
        raise ValueError("a Kv4Pool expected")
    check_pool(p, pool)


def _check(fn: str, st: int):
    if st != SKV_OK:
        raise SkvError(fn, st)


@dataclass
class Problem:
    """Python mirror of skv_problem (see include/skv.h for every field's meaning)."""

    batch: int
    n_kv_heads: int
    n_q_heads: int
    d_qk: int
    d_v: int
    max_len: int
    topk: int
    n_sink: int
    n_local: int
    block_size: int
    seq_lens: torch.Tensor  # device int32 [batch]
    d_idx: int = 0  # 0 -> d_qk
    n_idx_q_heads: int = 0  # 0 -> n_q_heads
    dtype: int = SKV_DTYPE_BF16
    group_agg: int = SKV_AGG_MEAN
    sm_scale: float = 0.0
    n_splits: int = 0

    def c(self) -> CProblem:
        return CProblem(self.batch, self.n_kv_heads, self.n_q_heads, self.d_qk, self.d_v,
                        self.d_idx or self.d_qk, self.n_idx_q_heads or self.n_q_heads, self.max_len,
                        self.topk, self.n_sink, self.n_local, self.block_size, self.dtype, self.group_agg,
                        float(self.sm_scale), self.n_splits,
                        None if self.seq_lens is None else self.seq_lens.data_ptr())


@dataclass
class Pool:
    """Python mirror of skv_kv_pool; tensors are [n_blocks, H, block_size, d].  With
    table_heads = 1 the table is [batch, H, stride] and the GPU pools [n_blocks, block_size, d].
    cached: a slot cache manages the GPU blocks (set when one is made for the pool)."""

    gpu_k: torch.Tensor
    gpu_v: Optional[torch.Tensor]
    slot_table: torch.Tensor  # device int32 [batch, stride], or [batch, H, stride] with table_heads = 1
    host_k: Optional[torch.Tensor] = None
    host_v: Optional[torch.Tensor] = None
    table_heads: int = 0
    cached: bool = False

    def c(self) -> CPool:
        return CPool(self.gpu_k.data_ptr(), None if self.gpu_v is None else self.gpu_v.data_ptr(),
                     self.gpu_k.shape[0],
                     None if self.host_k is None else self.host_k.data_ptr(),
                     None if self.host_v is None else self.host_v.data_ptr(),
                     0 if self.host_k is None else self.host_k.shape[0],
                     self.slot_table.data_ptr(), self.slot_table.shape[-1], self.table_heads)


@dataclass
class Kv4Pool(Pool):
    """A pool in 4 bits: uint8 tensors [n_blocks, H, block_size / 16, cell] (with table_heads = 1 the
    GPU ones [n_blocks, block_size / 16, cell]), cells as include/skv.h lays them out."""

    group: int = 32

    @staticmethod
    def cell_bytes(group: int) -> int:
        return 1024 + 64 * (128 // group)

    @classmethod
    def empty(cls, n_blocks: int, n_kv_heads: int, block_size: int, slot_table: torch.Tensor, group: int = 32,
              n_host_blocks: int = 0) -> "Kv4Pool":
        """Pools of n_blocks on the table's device (and n_host_blocks in pinned host memory)."""
        per_head = slot_table.dim() == 3
        cells = (block_size // 16, cls.cell_bytes(group))

        def make(n, heads, **kw):
            return torch.empty((n, *heads, *cells), dtype=torch.uint8, **kw) if n else None

        gpu = [make(n_blocks, () if per_head else (n_kv_heads,), device=slot_table.device) for _ in range(2)]
        host = [make(n_host_blocks, (n_kv_heads,), pin_memory=True) for _ in range(2)]
        return cls(*gpu, slot_table, *host, table_heads=int(per_head), group=group)

    def c(self) -> CPool:
        raise ValueError("a pool in 4 bits: the calls named *_kv4 take it")

    def c4(self) -> CPool:
        return super().c()

    def check(self, p: "Problem") -> None:
        """The pools' types and sizes, which the C side cannot see."""
        if self.group not in (32, 64, 128) or p.block_size % 16:
            raise ValueError("group: 32, 64 or 128; block_size: a multiple of 16")
        cells = p.block_size // 16 * self.cell_bytes(self.group)
        for name in ("gpu_k", "gpu_v", "host_k", "host_v"):
            t = getattr(self, name)
            if t is None and name.startswith("host"):
                continue
            heads = 1 if self.table_heads and name.startswith("gpu") else p.n_kv_heads
            if t is None or t.dtype != torch.uint8 or t.numel() != t.shape[0] * heads * cells or not t.is_contiguous():
                raise ValueError(f"{name}: contiguous uint8 blocks of {heads} x {cells} bytes expected")
        if self.gpu_v.shape[0] != self.gpu_k.shape[0] or (self.host_k is None) != (self.host_v is None) or (
                self.host_k is not None and self.host_v.shape[0] != self.host_k.shape[0]):
            raise ValueError("K and V pools of one size expected")


@dataclass
class IndexSrc:
    layout: int = SKV_INDEX_PAGED
    keys: Optional[torch.Tensor] = None

    def c(self) -> CIndex:
        return CIndex(self.layout, None if self.keys is None else self.keys.data_ptr())


def skv_workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t(0)
    cp = p.c()
    _check("skv_workspace_size", lib().skv_workspace_size(ctypes.byref(cp), ctypes.byref(n)))
    return n.value


def skv_score(p: Problem, q_score, index: IndexSrc, pool: Optional[Pool], scores, dev_status=None, stream=None):
    cp, ci = p.c(), index.c()
    cpool = pool.c() if pool is not None else None
    _check("skv_score", lib().skv_score(ctypes.byref(cp), _ptr(q_score), ctypes.byref(ci),
                                        ctypes.byref(cpool) if cpool is not None else None, _ptr(scores),
                                        _ptr(dev_status), _stream(stream)))


def skv_topk(p: Problem, scores, idx, ws, dev_status=None, stream=None):
    cp = p.c()
    _check("skv_topk", lib().skv_topk(ctypes.byref(cp), _ptr(scores), _ptr(idx), _ptr(ws),
                                      ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def skv_gather(p: Problem, pool: Pool, idx, k_out, v_out=None, dev_status=None, stream=None):
    cp, cpool = p.c(), pool.c()
    _check("skv_gather", lib().skv_gather(ctypes.byref(cp), ctypes.byref(cpool), _ptr(idx), _ptr(k_out),
                                          _ptr(v_out), _ptr(dev_status), _stream(stream)))


def skv_sparse_attn(p: Problem, q, pool: Pool, idx, out, lse, ws, dev_status=None, stream=None):
    cp, cpool = p.c(), pool.c()
    _check("skv_sparse_attn", lib().skv_sparse_attn(
        ctypes.byref(cp), _ptr(q), ctypes.byref(cpool), _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def skv_decode_step(p: Problem, q, q_score, index: IndexSrc, pool: Pool, scores, idx, out, lse, ws,
                    dev_status=None, stream=None):
    cp, ci, cpool = p.c(), index.c(), pool.c()
    _check("skv_decode_step", lib().skv_decode_step(
        ctypes.byref(cp), _ptr(q), _ptr(q_score), ctypes.byref(ci), ctypes.byref(cpool), _ptr(scores),
        _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


def skv_block_workspace_size(p: Problem, topk_blocks: int) -> tuple[int, int]:
    """(workspace bytes, attended-list length) of the block-selection calls."""
    n, ln = ctypes.c_size_t(0), ctypes.c_int32(0)
    cp = p.c()
    _check("skv_block_workspace_size", lib().skv_block_workspace_size(ctypes.byref(cp), int(topk_blocks),
                                                                      ctypes.byref(n), ctypes.byref(ln)))
    return n.value, ln.value


def skv_block_summaries(p: Problem, pool: Pool, summaries, dev_status=None, stream=None):
    cp, cpool = p.c(), pool.c()
    _check("skv_block_summaries", lib().skv_block_summaries(ctypes.byref(cp), ctypes.byref(cpool), _ptr(summaries),
                                                            _ptr(dev_status), _stream(stream)))


def skv_block_select(p: Problem, topk_blocks: int, q, summaries, block_idx, att_idx, ws, dev_status=None,
                     stream=None):
    cp = p.c()
    _check("skv_block_select", lib().skv_block_select(
        ctypes.byref(cp), int(topk_blocks), _ptr(q), _ptr(summaries), _ptr(block_idx), _ptr(att_idx), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def skv_block_decode_step(p: Problem, topk_blocks: int, q, summaries, pool: Pool, block_idx, att_idx, out, lse,
                          ws, dev_status=None, stream=None):
    cp, cpool = p.c(), pool.c()
    _check("skv_block_decode_step", lib().skv_block_decode_step(
        ctypes.byref(cp), int(topk_blocks), _ptr(q), _ptr(summaries), ctypes.byref(cpool), _ptr(block_idx),
        _ptr(att_idx), _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


@dataclass
class Prefetch:
    """Threshold-prefetch state (persistent across steps); see skv_prefetch in include/skv.h."""

    tau_ema: torch.Tensor   # float32 [rows], NaN to start
    epoch: torch.Tensor     # int32 [1] (uint32 on the device), 0 to start
    map: torch.Tensor       # int64 [rows * max_len], 0 to start
    staging: torch.Tensor   # [rows, cap, d_qk] of the pool's dtype
    count: torch.Tensor     # int32 [rows], 0 to start
    stats: Optional[torch.Tensor] = None  # int32 [2]
    alpha: float = 0.5

    @classmethod
    def new(cls, p: "Problem", cap: int, dtype: torch.dtype, device, alpha: float = 0.5,
            paged: bool = False) -> "Prefetch":
        """paged: a pool with separate V rows, whose staging holds the K rows, then the V rows."""
        rows = p.batch * p.n_kv_heads
        shape = (2, rows, max(cap, 1), p.d_qk) if paged else (rows, max(cap, 1), p.d_qk)
        return cls(tau_ema=torch.full((rows,), float("nan"), dtype=torch.float32, device=device),
                   epoch=torch.zeros((1,), dtype=torch.int32, device=device),
                   map=torch.zeros((rows * p.max_len,), dtype=torch.int64, device=device),
                   staging=torch.empty(shape, dtype=dtype, device=device),
                   count=torch.zeros((rows,), dtype=torch.int32, device=device),
                   stats=torch.zeros((2,), dtype=torch.int32, device=device), alpha=alpha)

    def c(self, cap: int, stats: bool = True) -> CPrefetch:
        st = self.stats.data_ptr() if (stats and self.stats is not None) else None
        return CPrefetch(self.tau_ema.data_ptr(), self.epoch.data_ptr(), self.map.data_ptr(), self.staging.data_ptr(),
                         self.count.data_ptr(), st, int(cap), float(self.alpha))


def skv_decode_step_prefetch(p: Problem, q, q_score, index: IndexSrc, pool: Pool, scores, idx, out, lse, ws,
                             pf: Prefetch, dev_status=None, stream=None, stats: bool = True):
    cp, ci, cpool, cpf = p.c(), index.c(), pool.c(), pf.c(pf.staging.shape[-2], stats)  # [..., cap, d]
    _check("skv_decode_step_prefetch", lib().skv_decode_step_prefetch(
        ctypes.byref(cp), _ptr(q), _ptr(q_score), ctypes.byref(ci), ctypes.byref(cpool), _ptr(scores), _ptr(idx),
        _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(cpf), _ptr(dev_status),
        _stream(stream)))


@dataclass
class SlotCache:
    """GPU slot-cache state (persistent across steps); see skv_slot_cache in include/skv.h."""

    owner: torch.Tensor   # int32 [n_gpu]
    prio: torch.Tensor    # int32 [n_gpu]
    step: torch.Tensor    # int32 [1]
    budget: int
    ws: torch.Tensor      # uint8: the update's own workspace
    stats: torch.Tensor   # int64 [3]: hits, misses, promotions summed over steps
    count: bool = True    # False: the update leaves stats untouched

    @classmethod
    def from_table(cls, p: "Problem", pool: "Pool", budget: int) -> "SlotCache":
        """Owners as the slot table names them, every slot unused so far."""
        cp, cpool = p.c(), pool.c()
        n = pool.gpu_k.shape[0]
        dev = pool.gpu_k.device
        owner = torch.full((n,), -1, dtype=torch.int64, device=dev)
        if pool.table_heads:  # one row per (request, KV head): owners (b * H + h) * stride + block
            t = pool.slot_table.reshape(-1).to(torch.int64)
            m = t >= 0
            owner[t[m]] = torch.arange(t.numel(), device=dev)[m]
        else:  # the latent layout's per-token map: owners b * max_len + position
            t = pool.slot_table[:, : p.max_len].to(torch.int64)
            b = torch.arange(t.shape[0], device=dev)[:, None].expand_as(t)
            pos = torch.arange(p.max_len, device=dev)[None, :].expand_as(t)
            m = t >= 0
            owner[t[m]] = (b[m] * p.max_len + pos[m])
        nb = ctypes.c_size_t(0)
        _check("skv_cache_prepare", lib().skv_cache_prepare())
        _check("skv_cache_workspace_size", lib().skv_cache_workspace_size(ctypes.byref(cp), ctypes.byref(cpool),
                                                                          int(budget), ctypes.byref(nb)))
        pool.cached = True  # appends keep the host rows behind its slots from now on
        return cls(owner=owner.to(torch.int32), prio=torch.full((n,), -1, dtype=torch.int32, device=dev),
                   step=torch.zeros((1,), dtype=torch.int32, device=dev), budget=int(budget),
                   ws=torch.empty((max(nb.value, 16),), dtype=torch.uint8, device=dev),
                   stats=torch.zeros((3,), dtype=torch.int64, device=dev))

    def c(self) -> CSlotCache:
        return CSlotCache(self.owner.data_ptr(), self.prio.data_ptr(), self.step.data_ptr(), self.budget,
                          self.stats.data_ptr() if self.count else None)


def skv_decode_step_cached(p: Problem, q, q_score, index: IndexSrc, pool: Pool, scores, idx, out, lse, ws,
                           cache: SlotCache, dev_status=None, stream=None):
    cp, ci, cpool, cc = p.c(), index.c(), pool.c(), cache.c()
    _check("skv_decode_step_cached", lib().skv_decode_step_cached(
        ctypes.byref(cp), _ptr(q), _ptr(q_score), ctypes.byref(ci), ctypes.byref(cpool), _ptr(scores), _ptr(idx),
        _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(cc), _ptr(cache.ws),
        cache.ws.numel(), _ptr(dev_status), _stream(stream)))


def skv_cache_update(p: Problem, pool: Pool, idx, ws, cache: SlotCache, dev_status=None, stream=None):
    cp, cpool, cc = p.c(), pool.c(), cache.c()
    _check("skv_cache_update", lib().skv_cache_update(
        ctypes.byref(cp), ctypes.byref(cpool), _ptr(idx), _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(cc),
        _ptr(cache.ws), cache.ws.numel(), _ptr(dev_status), _stream(stream)))


@dataclass
class Paris:
    """ParisKV retrieval parameters (skv_paris) and the per-row index it reads (skv_paris_index)."""

    signs: torch.Tensor          # device int8 [128]
    cent: torch.Tensor           # device uint8 [rows, max_len, 16]
    rec: torch.Tensor            # device int32 [rows, max_len, 32]: 16 code words, 16 fp32 weights
    hist: torch.Tensor           # device int32 [rows, 16, 256]
    beta_pm: int = 50
    rho_pm: int = 100
    m: int = 8

    @classmethod
    def new(cls, p: "Problem", signs: torch.Tensor, beta_pm: int = 50, rho_pm: int = 100) -> "Paris":
        rows, dev = p.batch * p.n_kv_heads, signs.device
        return cls(signs=signs, beta_pm=beta_pm, rho_pm=rho_pm,
                   cent=torch.zeros((rows, p.max_len, 16), dtype=torch.uint8, device=dev),
                   rec=torch.zeros((rows, p.max_len, 32), dtype=torch.int32, device=dev),
                   hist=torch.empty((rows, 16, 256), dtype=torch.int32, device=dev))

    @property
    def code(self) -> torch.Tensor:
        """[rows, max_len, 16] code words (a view of the records)."""
        return self.rec[..., :16]

    @property
    def w(self) -> torch.Tensor:
        """[rows, max_len, 16] fp32 weights (a view of the records)."""
        return self.rec[..., 16:].view(torch.float32)

    def c(self) -> CParis:
        return CParis(self.m, self.beta_pm, self.rho_pm, self.signs.data_ptr())

    def c_index(self) -> CParisIndex:
        return CParisIndex(self.cent.data_ptr(), self.rec.data_ptr(), self.hist.data_ptr())


def skv_paris_quantizer(m: int = 8):
    lv, th = (ctypes.c_float * 8)(), (ctypes.c_float * 7)()
    _check("skv_paris_quantizer", lib().skv_paris_quantizer(int(m), ctypes.cast(lv, ctypes.c_void_p),
                                                            ctypes.cast(th, ctypes.c_void_p)))
    return list(lv), list(th)


def skv_paris_encode(p: Problem, paris: Paris, index: IndexSrc, pool: Pool, dev_status=None, stream=None):
    cp, cpr, ci, cpool, cix = p.c(), paris.c(), index.c(), pool.c(), paris.c_index()
    _check("skv_paris_encode", lib().skv_paris_encode(ctypes.byref(cp), ctypes.byref(cpr), ctypes.byref(ci),
                                                      ctypes.byref(cpool), ctypes.byref(cix), _ptr(dev_status),
                                                      _stream(stream)))


def skv_paris_workspace_size(p: Problem, paris: Paris) -> int:
    n = ctypes.c_size_t(0)
    cp, cpr = p.c(), paris.c()
    _check("skv_paris_workspace_size", lib().skv_paris_workspace_size(ctypes.byref(cp), ctypes.byref(cpr),
                                                                      ctypes.byref(n)))
    return n.value


def skv_paris_workspace_offsets(p: Problem, paris: Paris) -> list:
    out = (ctypes.c_int64 * 9)()
    cp, cpr = p.c(), paris.c()
    _check("skv_paris_workspace_offsets", lib().skv_paris_workspace_offsets(
        ctypes.byref(cp), ctypes.byref(cpr), ctypes.cast(out, ctypes.c_void_p)))
    return list(out)


def skv_paris_select(p: Problem, paris: Paris, q_score, index: IndexSrc, pool: Pool, idx, ws, dev_status=None,
                     stream=None):
    cp, cpr, ci, cpool, cix = p.c(), paris.c(), index.c(), pool.c(), paris.c_index()
    _check("skv_paris_select", lib().skv_paris_select(
        ctypes.byref(cp), ctypes.byref(cpr), _ptr(q_score), ctypes.byref(ci), ctypes.byref(cix), ctypes.byref(cpool),
        _ptr(idx), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def skv_paris_decode_step(p: Problem, paris: Paris, q, q_score, index: IndexSrc, pool: Pool, idx, out, lse, ws,
                          dev_status=None, stream=None):
    cp, cpr, ci, cpool, cix = p.c(), paris.c(), index.c(), pool.c(), paris.c_index()
    _check("skv_paris_decode_step", lib().skv_paris_decode_step(
        ctypes.byref(cp), ctypes.byref(cpr), _ptr(q), _ptr(q_score), ctypes.byref(ci), ctypes.byref(cix),
        ctypes.byref(cpool), _ptr(idx), _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(),
        _ptr(dev_status), _stream(stream)))


@dataclass
class Rotary:
    """Norm and rotation of a model's queries and keys; see skv_rotary in include/skv.h."""

    inv_freq: Optional[torch.Tensor]        # device float32 [rot_dim / 2]; None with rot_dim 0
    rot_dim: int = 0
    rot_start: int = 0
    style: int = SKV_ROPE_HALF
    norm_dim: int = 0                       # 0: the whole row
    eps: float = 1e-6
    q_gamma: Optional[torch.Tensor] = None  # device [norm_dim] of the element type; None: not normed
    k_gamma: Optional[torch.Tensor] = None

    def check(self, p: Problem) -> None:
        """The tensors' types, sizes and devices, which the C side cannot see."""
        same_device(p, inv_freq=self.inv_freq, q_gamma=self.q_gamma, k_gamma=self.k_gamma)
        if self.rot_dim and (self.inv_freq is None or self.inv_freq.dtype != torch.float32
                             or self.inv_freq.numel() != self.rot_dim // 2 or not self.inv_freq.is_contiguous()):
            raise ValueError("inv_freq: contiguous float32 [rot_dim / 2]")
        for g in (self.q_gamma, self.k_gamma):
            if g is not None and (g.dtype != element_type(p) or g.numel() != (self.norm_dim or p.d_qk)
                                  or not g.is_contiguous()):
                raise ValueError("gamma: contiguous [norm_dim] of the element type")

    def c(self) -> CRotary:
        return CRotary(self.rot_start, self.rot_dim, self.style, self.norm_dim, float(self.eps),
                       None if self.inv_freq is None else self.inv_freq.data_ptr(),
                       None if self.q_gamma is None else self.q_gamma.data_ptr(),
                       None if self.k_gamma is None else self.k_gamma.data_ptr())


def element_type(p: Problem) -> torch.dtype:
    return torch.float32 if p.dtype == SKV_DTYPE_F32 else torch.bfloat16


def _rows(name: str, t: Optional[torch.Tensor], n: int, heads: int, d: int, dtype: torch.dtype):
    """(pointer, token stride) of [n, heads, d] rows whose heads are packed."""
    if t is None:
        return None, 0
    if t.dtype != dtype or t.dim() != 3 or t.shape[0] != n or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name}: {dtype} [{n}, {heads}, {d}] expected, got {t.dtype} {tuple(t.shape)}")
    st = t.stride()
    if (st[2] != 1 and d > 1) or (st[1] != d and heads > 1):
        raise ValueError(f"{name}: a token's heads must be packed")
    return t.data_ptr(), st[0]


def _ids(name: str, t: Optional[torch.Tensor], n: int):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 [{n}] expected")
    return t.data_ptr()


def c_tokens(p: Problem, q, k, v, positions, requests) -> CTokens:
    """skv_tokens of [n, heads, d] tensors (column ranges of a fused projection included)."""
    first = k if k is not None else q
    if first is None:
        raise ValueError("q or k is needed")
    n, dtype = first.shape[0], element_type(p)
    if n >= 2 ** 31:
        raise ValueError("at most 2^31 - 1 tokens")
    check_lens(p)
    same_device(p, q=q, k=k, v=v, positions=positions, requests=requests)
    qp, qs = _rows("q", q, n, p.n_q_heads, p.d_qk, dtype)
    kp, ks = _rows("k", k, n, p.n_kv_heads, p.d_qk, dtype)
    vp, vs = _rows("v", v, n, p.n_kv_heads, p.d_v, dtype)
    return CTokens(n, 0, qp, kp, vp, qs, ks, vs, _ids("positions", positions, n), _ids("requests", requests, n))


def _out_rows(name: str, out, src, heads: int, d: int, dtype: torch.dtype):
    """Pointer of an output: packed rows, or the input itself (in place at its stride)."""
    if out is None:
        return None
    if src is None or out.device != src.device:
        raise ValueError(f"{name}: an output needs its input, on the same device")
    _, stride = _rows(name, out, src.shape[0], heads, d, dtype)
    if src.shape[0] > 1 and stride != (src.stride(0) if out.data_ptr() == src.data_ptr() else heads * d):
        raise ValueError(f"{name}: packed rows, or the input itself")
    return out.data_ptr()


def skv_qk_norm_rope(p: Problem, rotary: Rotary, q, k, q_out, k_out, positions=None, requests=None, dev_status=None,
                     stream=None):
    rotary.check(p)
    same_device(p, dev_status=dev_status)
    cp, cr, ct = p.c(), rotary.c(), c_tokens(p, q, k, None, positions, requests)
    qo = _out_rows("q_out", q_out, q, p.n_q_heads, p.d_qk, element_type(p))
    ko = _out_rows("k_out", k_out, k, p.n_kv_heads, p.d_qk, element_type(p))
    _check("skv_qk_norm_rope", lib().skv_qk_norm_rope(ctypes.byref(cp), ctypes.byref(cr), ctypes.byref(ct), qo, ko,
                                                      _ptr(dev_status), raw_stream(p.seq_lens.get_device(), stream)))


def _append(fn: str, p: Problem, rotary: Rotary, q, k, v, pool: Pool, q_out, positions, requests, dev_status, stream):
    rotary.check(p)
    check_pool(p, pool)
    same_device(p, dev_status=dev_status)
    cp, cr, ct, cpool = p.c(), rotary.c(), c_tokens(p, q, k, v, positions, requests), pool.c()
    qo = _out_rows("q_out", q_out, q, p.n_q_heads, p.d_qk, element_type(p))
    _check(fn, getattr(lib(), fn)(ctypes.byref(cp), ctypes.byref(cr), ctypes.byref(ct), ctypes.byref(cpool), qo,
                                  _ptr(dev_status), raw_stream(p.seq_lens.get_device(), stream)))


def skv_append_kv(p: Problem, rotary: Rotary, q, k, v, pool: Pool, q_out, positions=None, requests=None,
                  dev_status=None, stream=None):
    if pool.cached:
        raise ValueError("a slot cache manages this pool: skv_append_kv_cached")
    _append("skv_append_kv", p, rotary, q, k, v, pool, q_out, positions, requests, dev_status, stream)


def skv_append_kv_cached(p: Problem, rotary: Rotary, q, k, v, pool: Pool, q_out, positions=None, requests=None,
                         dev_status=None, stream=None):
    _append("skv_append_kv_cached", p, rotary, q, k, v, pool, q_out, positions, requests, dev_status, stream)


def skv_append_kv4(p: Problem, rotary: Rotary, q, k, v, pool: Kv4Pool, q_out, positions=None, requests=None,
                   dev_status=None, stream=None):
    rotary.check(p)
    check_pool4(p, pool)
    same_device(p, dev_status=dev_status)
    cp, cr, ct, cpool = p.c(), rotary.c(), c_tokens(p, q, k, v, positions, requests), pool.c4()
    qo = _out_rows("q_out", q_out, q, p.n_q_heads, p.d_qk, element_type(p))
    _check("skv_append_kv4", lib().skv_append_kv4(
        ctypes.byref(cp), ctypes.byref(cr), ctypes.byref(ct), ctypes.byref(cpool), pool.group, qo, _ptr(dev_status),
        raw_stream(p.seq_lens.get_device(), stream)))


def dense(p: Problem, name: str, t, dtype, shape) -> None:
    """A tensor's type, shape, layout and device (None passes)."""
    if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous()
                          or t.device != p.seq_lens.device):
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on {p.seq_lens.device} expected")


def list_heads(p: Problem) -> int:
    """Rows of scores and lists a request: per KV head, or per query head under SKV_AGG_HEAD."""
    return p.n_q_heads if p.group_agg == SKV_AGG_HEAD else p.n_kv_heads


def skv_gather_kv4(p: Problem, pool: Kv4Pool, idx, k_out, v_out=None, dev_status=None, stream=None):
    check_pool4(p, pool)
    rows = (p.batch, list_heads(p))
    dense(p, "idx", idx, torch.int32, rows + (p.topk,))
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        dense(p, name, t, element_type(p), rows + (p.n_sink + p.topk + p.n_local, 128))
    device = same_device(p, dev_status=dev_status)
    cp, cpool = p.c(), pool.c4()
    _check("skv_gather_kv4", lib().skv_gather_kv4(
        ctypes.byref(cp), ctypes.byref(cpool), pool.group, _ptr(idx), _ptr(k_out), _ptr(v_out), _ptr(dev_status),
        raw_stream(device, stream)))


def skv_score_kv4(p: Problem, q_score, pool: Kv4Pool, scores, dev_status=None, stream=None):
    check_pool4(p, pool)
    dense(p, "q_score", q_score, torch.bfloat16, (p.batch, p.n_idx_q_heads or p.n_q_heads, 128))
    dense(p, "scores", scores, torch.float32, (p.batch, list_heads(p), p.max_len))
    device = same_device(p, dev_status=dev_status)
    cp, cpool = p.c(), pool.c4()
    _check("skv_score_kv4", lib().skv_score_kv4(ctypes.byref(cp), _ptr(q_score), ctypes.byref(cpool), pool.group,
                                                _ptr(scores), _ptr(dev_status), raw_stream(device, stream)))


def skv_kv4_workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t(0)
    cp = p.c()
    _check("skv_kv4_workspace_size", lib().skv_kv4_workspace_size(ctypes.byref(cp), ctypes.byref(n)))
    return n.value


def list_ptr(p: Problem, idx) -> Optional[int]:
    """A list's pointer: NULL means no list, so one of no entries (topk 0) gets another, never read."""
    return None if idx is None else (idx if idx.numel() else p.seq_lens).data_ptr()


def _attn_kv4(p: Problem, q, pool, idx, out, lse, ws, dev_status) -> int:
    check_pool4(p, pool)
    dense(p, "q", q, torch.bfloat16, (p.batch, p.n_q_heads, 128))
    dense(p, "idx", idx, torch.int32, (p.batch, list_heads(p), p.topk))
    dense(p, "out", out, torch.bfloat16, (p.batch, p.n_q_heads, 128))
    dense(p, "lse", lse, torch.float32, (p.batch, p.n_q_heads))
    return same_device(p, ws=ws, dev_status=dev_status)


def skv_attn_kv4(p: Problem, q, pool: Kv4Pool, idx, out, lse, ws, dev_status=None, stream=None):
    """idx None: over every position of each request's history."""
    device = _attn_kv4(p, q, pool, idx, out, lse, ws, dev_status)
    cp, cpool = p.c(), pool.c4()
    _check("skv_attn_kv4", lib().skv_attn_kv4(
        ctypes.byref(cp), _ptr(q), ctypes.byref(cpool), pool.group, list_ptr(p, idx), _ptr(out), _ptr(lse), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), raw_stream(device, stream)))


def skv_decode_step_kv4(p: Problem, q, q_score, pool: Kv4Pool, scores, idx, out, lse, ws, dev_status=None,
                        stream=None):
    device = _attn_kv4(p, q, pool, idx, out, lse, ws, dev_status)
    dense(p, "q_score", q_score, torch.bfloat16, (p.batch, p.n_idx_q_heads or p.n_q_heads, 128))
    dense(p, "scores", scores, torch.float32, (p.batch, list_heads(p), p.max_len))
    cp, cpool = p.c(), pool.c4()
    _check("skv_decode_step_kv4", lib().skv_decode_step_kv4(
        ctypes.byref(cp), _ptr(q), _ptr(q_score), ctypes.byref(cpool), pool.group, _ptr(scores), list_ptr(p, idx),
        _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status), raw_stream(device, stream)))


@dataclass
class Tables:
    """Block tables kept on the GPU; see skv_tables in include/skv.h.  seq_lens, batch, max_len and
    block_size are the problem's."""

    slot_table: torch.Tensor   # device int32 [batch, stride]
    free_blocks: torch.Tensor  # device int32 [n_blocks]: the stack, state[0] entries
    state: torch.Tensor        # device int32 [4]
    base: int = 0

    def check(self, p: Problem) -> None:
        check_lens(p)
        same_device(p, slot_table=self.slot_table, free_blocks=self.free_blocks, state=self.state)
        for name, n in (("slot_table", p.batch), ("free_blocks", 0), ("state", 4)):
            t = getattr(self, name)
            if t.dtype != torch.int32 or not t.is_contiguous() or t.shape[0] < n:
                raise ValueError(f"{name}: contiguous int32 expected")
        if self.slot_table.dim() != 2:
            raise ValueError("slot_table: [batch, stride], one row a request")

    def c(self, p: Problem) -> CTables:
        return CTables(p.batch, p.max_len, p.block_size, self.base, self.slot_table.shape[1],
                       self.free_blocks.numel(), self.slot_table.data_ptr(), p.seq_lens.data_ptr(),
                       self.free_blocks.data_ptr(), self.state.data_ptr())


def skv_update_tables(p: Problem, tables: Tables, n_new, n_tokens: int = 0, positions=None, requests=None, slots=None,
                      dev_status=None, stream=None):
    tables.check(p)
    dense(p, "n_new", n_new, torch.int32, (p.batch,))
    for name, t, dtype in (("positions", positions, torch.int32), ("requests", requests, torch.int32),
                           ("slots", slots, torch.int64)):
        dense(p, name, t, dtype, (n_tokens,))
    device = same_device(p, dev_status=dev_status)
    ct = tables.c(p)
    _check("skv_update_tables", lib().skv_update_tables(ctypes.byref(ct), _ptr(n_new), int(n_tokens), _ptr(positions),
                                                        _ptr(requests), _ptr(slots), _ptr(dev_status),
                                                        raw_stream(device, stream)))


@dataclass
class Prefix:
    """The positions a batch shares; see skv_prefix in include/skv.h."""

    table: Optional[torch.Tensor]  # device int32 [ceil(len / block_size)]; None with len 0
    len: int

    def check(self, p: Problem) -> None:
        if not 0 <= self.len <= p.max_len:
            raise ValueError(f"prefix length {self.len} outside [0, {p.max_len}]")
        same_device(p, table=self.table)
        need = (self.len + p.block_size - 1) // p.block_size
        if need and (self.table is None or self.table.dtype != torch.int32 or self.table.numel() < need
                     or not self.table.is_contiguous()):
            raise ValueError(f"prefix table: contiguous int32 [{need}] expected")

    def c(self) -> CPrefix:
        return CPrefix(None if self.table is None else self.table.data_ptr(), int(self.len), 0)


def skv_prefix_workspace_size(p: Problem, prefix_len: int) -> int:
    n = ctypes.c_size_t(0)
    cp = p.c()
    _check("skv_prefix_workspace_size", lib().skv_prefix_workspace_size(ctypes.byref(cp), int(prefix_len),
                                                                        ctypes.byref(n)))
    return n.value


def skv_prefix_attn(p: Problem, q, pool: Pool, prefix: Prefix, out, lse, ws, dev_status=None, stream=None):
    prefix.check(p)
    check_pool(p, pool)
    shape = (p.batch, p.n_q_heads)
    for name, t, dtype, want in (("q", q, torch.bfloat16, shape + (p.d_qk,)), ("out", out, torch.bfloat16, shape + (p.d_v,)),
                                 ("lse", lse, torch.float32, shape)):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != want or not t.is_contiguous()):
            raise ValueError(f"{name}: contiguous {dtype} {list(want)} expected")
    device = same_device(p, q=q, out=out, lse=lse, ws=ws, dev_status=dev_status)
    cp, cpool, cx = p.c(), pool.c(), prefix.c()
    _check("skv_prefix_attn", lib().skv_prefix_attn(
        ctypes.byref(cp), _ptr(q), ctypes.byref(cpool), ctypes.byref(cx), _ptr(out), _ptr(lse), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), raw_stream(device, stream)))


def skv_status_string(status: int) -> str:
    return lib().skv_status_string(status).decode()


def skv_launch_count() -> int:
    return int(lib().skv_launch_count())


def skv_check_wait_timeout(limit_cycles: int, arrive: int, dev_status, stream=None):
    _check("skv_check_wait_timeout", lib().skv_check_wait_timeout(int(limit_cycles), int(arrive), _ptr(dev_status),
                                                                  _stream(stream)))
