"""DecodeStep: owns the output and workspace tensors of one decode step and calls the C ABI.

A thin convenience over the binding: it allocates (with torch) the scores,
index, output, lse, workspace and status buffers once, then every `run()` is a
single skv_decode_step call enqueued on the current stream.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B


class DecodeStep:
    def __init__(self, problem: B.Problem, pool: B.Pool, q: torch.Tensor, index: B.IndexSrc,
                 q_score: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None):
        self.p = problem
        self.pool = pool
        self.q = q
        self.q_score = q_score
        self.index = index
        dev = q.device
        # one selection row per KV head, or per query head under the per-head reading
        sel_heads = problem.n_q_heads if problem.group_agg == B.SKV_AGG_HEAD else problem.n_kv_heads
        rows = problem.batch * sel_heads
        self.scores = torch.empty((problem.batch, sel_heads, problem.max_len), dtype=torch.float32, device=dev)
        self.idx = torch.empty((problem.batch, sel_heads, max(problem.topk, 1)), dtype=torch.int32, device=dev)
        self.out = torch.empty((problem.batch, problem.n_q_heads, problem.d_v), dtype=out_dtype or q.dtype,
                               device=dev)
        self.lse = torch.empty((problem.batch, problem.n_q_heads), dtype=torch.float32, device=dev)
        ws_bytes = B.skv_workspace_size(problem)
        self.ws = torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        assert rows > 0

    def run(self, stream=None):
        B.skv_decode_step(self.p, self.q, self.q_score, self.index, self.pool, self.scores, self.idx, self.out,
                          self.lse, self.ws, self.status, stream)

    def enable_prefetch(self, cap: int, alpha: float = 0.5):
        """Fresh threshold-prefetch state for run_prefetch() (latent layout, or a paged pool with
        contiguous index keys)."""
        self.pf = B.Prefetch.new(self.p, cap, self.pool.gpu_k.dtype, self.q.device, alpha,
                                 paged=self.pool.gpu_v is not None)
        return self.pf

    def run_prefetch(self, stream=None, stats: bool = True):
        """One step with threshold prefetch; stats=False leaves the staged/read counters untouched."""
        B.skv_decode_step_prefetch(self.p, self.q, self.q_score, self.index, self.pool, self.scores, self.idx,
                                   self.out, self.lse, self.ws, self.pf, self.status, stream, stats=stats)

    def enable_cache(self, budget: int):
        """Switch to skv_decode_step_cached: the GPU slot pool becomes a managed cache (the latent
        layout, or K/V pools with one table row per (request, KV head))."""
        self.cache = B.SlotCache.from_table(self.p, self.pool, budget)
        return self.cache

    def run_cached(self, stream=None):
        B.skv_decode_step_cached(self.p, self.q, self.q_score, self.index, self.pool, self.scores, self.idx, self.out,
                                 self.lse, self.ws, self.cache, self.status, stream)

    def cache_update(self, stream=None):
        """The slot-cache update alone, for the step run() just enqueued."""
        B.skv_cache_update(self.p, self.pool, self.idx, self.ws, self.cache, self.status, stream)

    def score(self, stream=None):
        B.skv_score(self.p, self.q_score if self.q_score is not None else self.q, self.index, self.pool,
                    self.scores, self.status, stream)

    def topk(self, stream=None):
        B.skv_topk(self.p, self.scores, self.idx, self.ws, self.status, stream)

    def attend(self, stream=None):
        B.skv_sparse_attn(self.p, self.q, self.pool, self.idx, self.out, self.lse, self.ws, self.status, stream)

    @classmethod
    def from_workload(cls, wl, n_splits: int = 0, sm_scale: Optional[float] = None, group_agg: int = B.SKV_AGG_MEAN):
        """Build from an object with the seeded generator's attribute names (duck-typed)."""
        dtype = B.SKV_DTYPE_F32 if wl.dtype == torch.float32 else B.SKV_DTYPE_BF16
        contig = getattr(wl, "index_keys", None) is not None
        q_score = wl.q_idx if contig else None
        p = B.Problem(batch=wl.B, n_kv_heads=wl.H, n_q_heads=wl.Hq, d_qk=wl.d_qk, d_v=wl.d_v, max_len=wl.L,
                      topk=wl.k, n_sink=wl.ns, n_local=wl.nl, block_size=wl.bs, seq_lens=wl.seq_lens,
                      d_idx=wl.d_idx, n_idx_q_heads=(q_score.shape[1] if contig else wl.Hq), dtype=dtype,
                      sm_scale=float(sm_scale if sm_scale is not None else wl.sm_scale), n_splits=n_splits,
                      group_agg=group_agg)
        pool = B.Pool(wl.gpu_k, wl.gpu_v, wl.table, wl.host_k, wl.host_v)
        index = B.IndexSrc(B.SKV_INDEX_CONTIG, wl.index_keys) if contig else B.IndexSrc(B.SKV_INDEX_PAGED)
        return cls(p, pool, wl.q, index, q_score=q_score)


class BlockStep:
    """Block-selection decode (per-block key summaries): owns the summaries, the
    chosen blocks, the attended list, the output and the workspace; `summarize()`
    is the maintenance call, `run()` one skv_block_decode_step."""

    def __init__(self, problem: B.Problem, pool: B.Pool, q: torch.Tensor, topk_blocks: int):
        self.p = problem
        self.pool = pool
        self.q = q
        self.K = int(topk_blocks)
        dev = q.device
        nb = (problem.max_len + 15) // 16
        self.summaries = torch.empty((problem.batch, problem.n_kv_heads, nb, 2, problem.d_qk),
                                     dtype=pool.gpu_k.dtype, device=dev)
        ws_bytes, self.list_len = B.skv_block_workspace_size(problem, self.K)
        self.block_idx = torch.empty((problem.batch, problem.n_kv_heads, max(self.K, 1)), dtype=torch.int32,
                                     device=dev)
        self.att_idx = torch.empty((problem.batch, problem.n_kv_heads, max(self.list_len, 1)), dtype=torch.int32,
                                   device=dev)
        self.out = torch.empty((problem.batch, problem.n_q_heads, problem.d_v), dtype=q.dtype, device=dev)
        self.lse = torch.empty((problem.batch, problem.n_q_heads), dtype=torch.float32, device=dev)
        self.ws = torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)

    def summarize(self, stream=None):
        B.skv_block_summaries(self.p, self.pool, self.summaries, self.status, stream)

    def select(self, stream=None):
        B.skv_block_select(self.p, self.K, self.q, self.summaries, self.block_idx, self.att_idx, self.ws,
                           self.status, stream)

    def run(self, stream=None):
        B.skv_block_decode_step(self.p, self.K, self.q, self.summaries, self.pool, self.block_idx, self.att_idx,
                                self.out, self.lse, self.ws, self.status, stream)

    @classmethod
    def from_workload(cls, wl, topk_blocks: int, group_agg: int = B.SKV_AGG_MEAN, n_splits: int = 0):
        """Build from a paged workload of the seeded generator (duck-typed attribute names)."""
        dtype = B.SKV_DTYPE_F32 if wl.dtype == torch.float32 else B.SKV_DTYPE_BF16
        p = B.Problem(batch=wl.B, n_kv_heads=wl.H, n_q_heads=wl.Hq, d_qk=wl.d_qk, d_v=wl.d_v, max_len=wl.L,
                      topk=topk_blocks, n_sink=wl.ns, n_local=wl.nl, block_size=wl.bs, seq_lens=wl.seq_lens,
                      d_idx=wl.d_qk, n_idx_q_heads=wl.Hq, dtype=dtype, sm_scale=float(wl.sm_scale),
                      n_splits=n_splits, group_agg=group_agg)
        pool = B.Pool(wl.gpu_k, wl.gpu_v, wl.table, wl.host_k, wl.host_v)
        return cls(p, pool, wl.q, topk_blocks)


class ParisStep:
    """ParisKV retrieval decode (skv_paris_decode_step): owns the index, the selection, the
    output and the workspace; `encode()` builds the index from the keys (maintenance),
    `run()` is one step."""

    def __init__(self, step: DecodeStep, signs: torch.Tensor, beta_pm: int = 50, rho_pm: int = 100):
        self.p, self.pool, self.q, self.q_score, self.index = step.p, step.pool, step.q, step.q_score, step.index
        self.paris = B.Paris.new(self.p, signs, beta_pm, rho_pm)
        self.idx, self.out, self.lse, self.status = step.idx, step.out, step.lse, step.status
        n = B.skv_paris_workspace_size(self.p, self.paris)
        self.ws = torch.empty((max(n, 16),), dtype=torch.uint8, device=signs.device)
        self.offsets = B.skv_paris_workspace_offsets(self.p, self.paris)

    @classmethod
    def from_workload(cls, wl, signs: torch.Tensor, beta_pm: int = 50, rho_pm: int = 100, n_splits: int = 0):
        return cls(DecodeStep.from_workload(wl, n_splits=n_splits), signs, beta_pm, rho_pm)

    def encode(self, stream=None):
        B.skv_paris_encode(self.p, self.paris, self.index, self.pool, self.status, stream)

    def run(self, stream=None):
        B.skv_paris_decode_step(self.p, self.paris, self.q, self.q_score, self.index, self.pool, self.idx,
                                self.out, self.lse, self.ws, self.status, stream)

    def select(self, stream=None):
        """The retrieval alone: the selection into idx."""
        B.skv_paris_select(self.p, self.paris, self.q_score if self.q_score is not None else self.q, self.index,
                           self.pool, self.idx, self.ws, self.status, stream)

    def attend(self, stream=None):
        """The attention alone over the current selection (same workspace)."""
        B.skv_sparse_attn(self.p, self.q, self.pool, self.idx, self.out, self.lse, self.ws, self.status, stream)

    def view(self, name: str) -> torch.Tensor:
        """A workspace intermediate: qt, nq, W, S, cand_len, cand, cand_score, sim."""
        rows, c_cap, L = self.p.batch * self.p.n_kv_heads, self.offsets[7], self.p.max_len
        k = ("qt", "nq", "W", "S", "cand_len", "cand", "cand_score", None, "sim").index(name)
        shape, dt = {"qt": ((rows, 128), torch.float32), "nq": ((rows,), torch.float32),
                     "W": ((rows, 16, 256), torch.uint8), "S": ((rows, L), torch.uint8),
                     "sim": ((rows, 16, 256), torch.float32),
                     "cand_len": ((self.p.batch,), torch.int32), "cand": ((rows, c_cap), torch.int32),
                     "cand_score": ((rows, c_cap), torch.float32)}[name]
        n = int(torch.tensor(shape).prod().item()) * torch.tensor([], dtype=dt).element_size()
        return self.ws[self.offsets[k]: self.offsets[k] + n].view(dt).view(shape)


class TokenStep:
    """New tokens of a layer: `norm_rope()` norms and rotates queries and keys, `append()` also
    writes keys and values to the pool.  The problem, the rotary parameters and the pool are
    marshalled once, here; every call marshals only its tokens.  Status bits add up in `status`.
    Other tensors in their places need a new step; the marshalled ones live as long as this one.
    Appends to a pool with a slot cache (`pool.cached`) keep the host rows behind its slots current."""

    def __init__(self, problem: B.Problem, rotary: B.Rotary, pool: Optional[B.Pool] = None):
        rotary.check(problem)
        if pool is not None:
            B.check_pool(problem, pool)
        self.p, self.rotary, self.pool = problem, rotary, pool
        dev = problem.seq_lens.device
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._held = [*vars(problem).values(), *vars(rotary).values(), *(vars(pool).values() if pool else ())]
        self._p, self._r = ctypes.byref(problem.c()), ctypes.byref(rotary.c())
        self._pool = None if pool is None else ctypes.byref(pool.c())
        self._st = self.status.data_ptr()
        self._dtype = B.element_type(problem)
        self._norm_rope = B.lib().skv_qk_norm_rope
        self._append, self._append_cached = B.lib().skv_append_kv, B.lib().skv_append_kv_cached
        self._device = problem.seq_lens.get_device()
        self._seen = None  # the token layout that has been checked

    def _tokens(self, q, k, v, positions, requests, q_out, k_out):
        """skv_tokens and the outputs' pointers.  A layout -- types, shapes, strides, devices, what is in
        place -- is checked in full when it differs from the last one checked."""
        tensors = (q, k, v, positions, requests, q_out, k_out)
        ptr = [None if t is None else t.data_ptr() for t in tensors]
        seen = [None if t is None else (t.dtype, t.shape, t.stride(), t.get_device()) for t in tensors]
        seen.append(ptr[5] == ptr[0])
        seen.append(ptr[6] == ptr[1])
        if seen != self._seen:
            B.c_tokens(self.p, q, k, v, positions, requests)
            if q_out is not None:
                B._out_rows("q_out", q_out, q, self.p.n_q_heads, self.p.d_qk, self._dtype)
            if k_out is not None:
                B._out_rows("k_out", k_out, k, self.p.n_kv_heads, self.p.d_qk, self._dtype)
            self._seen = seen
        lq, lk, lv = seen[:3]
        return (B.CTokens((lk or lq)[1][0], 0, ptr[0], ptr[1], ptr[2], lq[2][0] if lq else 0, lk[2][0] if lk else 0,
                          lv[2][0] if lv else 0, ptr[3], ptr[4]), ptr[5], ptr[6])

    def _new(self, src, heads, stream):
        """An output, of the allocator's pool of the stream that writes it."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._new(src, heads, None)
        return torch.empty((src.shape[0], heads, self.p.d_qk), dtype=src.dtype, device=src.device)

    def norm_rope(self, q, k, positions=None, requests=None, q_out=None, k_out=None, stream=None):
        """(q_out, k_out): new tensors unless given; pass q and k themselves to work in place.
        Padding tokens' rows are not written."""
        if q_out is None and q is not None:
            q_out = self._new(q, self.p.n_q_heads, stream)
        if k_out is None and k is not None:
            k_out = self._new(k, self.p.n_kv_heads, stream)
        ct, qo, ko = self._tokens(q, k, None, positions, requests, q_out, k_out)
        st = self._norm_rope(self._p, self._r, ctypes.byref(ct), qo, ko, self._st, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_qk_norm_rope", st)
        return q_out, k_out

    def append(self, q, k, v, positions=None, requests=None, q_out=None, stream=None):
        """Appends k and v to the pool; returns q_out (None without q)."""
        if self._pool is None:
            raise ValueError("append() needs a pool")
        call = self._append_cached if self.pool.cached else self._append
        if q_out is None and q is not None:
            q_out = self._new(q, self.p.n_q_heads, stream)
        ct, qo, _ = self._tokens(q, k, v, positions, requests, q_out, None)
        st = call(self._p, self._r, ctypes.byref(ct), self._pool, qo, self._st, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_append_kv_cached" if self.pool.cached else "skv_append_kv", st)
        return q_out


class PrefixStep:
    """Attention of a batch over a shared prefix and every request's own tail: owns the output,
    lse, workspace and status; `run(q)` is one skv_prefix_attn.  The problem, the pool and the
    prefix are marshalled once, here; other tensors in their places need a new step, and the
    marshalled ones live as long as this one."""

    def __init__(self, problem: B.Problem, pool: B.Pool, prefix: B.Prefix):
        prefix.check(problem)
        self.p, self.pool, self.prefix = problem, pool, prefix
        B.check_pool(problem, pool)
        dev = problem.seq_lens.device
        self._device = problem.seq_lens.get_device()
        self._shape = (problem.batch, problem.n_q_heads, problem.d_qk)
        self._held = [*vars(problem).values(), *vars(pool).values(), *vars(prefix).values()]
        self._p, self._pool, self._prefix = (ctypes.byref(x.c()) for x in (problem, pool, prefix))
        self.out = torch.empty((problem.batch, problem.n_q_heads, problem.d_v), dtype=pool.gpu_k.dtype, device=dev)
        self.lse = torch.empty((problem.batch, problem.n_q_heads), dtype=torch.float32, device=dev)
        self.ws = torch.empty((max(B.skv_prefix_workspace_size(problem, prefix.len), 16),), dtype=torch.uint8,
                              device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._tail = (self.out.data_ptr(), self.lse.data_ptr(), self.ws.data_ptr(), self.ws.numel(),
                      self.status.data_ptr())
        self._call = B.lib().skv_prefix_attn

    def run(self, q, stream=None):
        """(out, lse), the step's own buffers."""
        if q.shape != self._shape or q.dtype != self.out.dtype or not q.is_contiguous() \
                or q.get_device() != self._device:
            raise ValueError(f"q: contiguous {self.out.dtype} {list(self._shape)} on {self.out.device} expected")
        st = self._call(self._p, q.data_ptr(), self._pool, self._prefix, *self._tail, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_prefix_attn", st)
        return self.out, self.lse
