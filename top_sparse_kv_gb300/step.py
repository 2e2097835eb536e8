"""DecodeStep: owns the output and workspace tensors of one decode step and calls the C ABI.

A thin convenience over the binding: it allocates (with torch) the scores,
index, output, lse, workspace and status buffers once, then every `run()` is a
single skv_decode_step call enqueued on the current stream.
"""

from __future__ import annotations

import contextlib
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
    Appends to a pool with a slot cache (`pool.cached`) keep the host rows behind its slots current;
    those to a Kv4Pool write 4 bits."""

    def __init__(self, problem: B.Problem, rotary: B.Rotary, pool: Optional[B.Pool] = None):
        rotary.check(problem)
        if pool is not None:
            B.check_pool(problem, pool)
        self._kv4 = (pool.group,) if isinstance(pool, B.Kv4Pool) else ()
        self.p, self.rotary, self.pool = problem, rotary, pool
        dev = problem.seq_lens.device
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._held = [*vars(problem).values(), *vars(rotary).values(), *(vars(pool).values() if pool else ())]
        self._p, self._r = ctypes.byref(problem.c()), ctypes.byref(rotary.c())
        self._pool = None if pool is None else ctypes.byref(pool.c4() if self._kv4 else pool.c())
        self._st = self.status.data_ptr()
        self._dtype = B.element_type(problem)
        self._norm_rope = B.lib().skv_qk_norm_rope
        self._append = B.lib().skv_append_kv4 if self._kv4 else B.lib().skv_append_kv
        self._append_cached = B.lib().skv_append_kv_cached
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
        st = call(self._p, self._r, ctypes.byref(ct), self._pool, *self._kv4, qo, self._st,
                  B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError(call.__name__, st)
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


class Kv4Step:
    """Decode over a pool in 4 bits: `score()`, `topk()`, `attend()` over a selection, `attend_all()`
    over whole histories, `gather()` of the attended rows' values, and `run()`, one
    skv_decode_step_kv4.  Owns scores, idx, out, lse, workspace and status; problem and pool are
    marshalled once, here, and live as long as the step."""

    def __init__(self, problem: B.Problem, pool: B.Kv4Pool):
        B.check_pool4(problem, pool)
        self.p, self.pool = problem, pool
        p, self._dev, lib = problem, problem.seq_lens.device, B.lib()
        self._device = p.seq_lens.get_device()
        self._held = [*vars(problem).values(), *vars(pool).values()]
        self._p, self._pool, self._group = ctypes.byref(p.c()), ctypes.byref(pool.c4()), pool.group
        heads = B.list_heads(p)
        self._q = torch.Size((p.batch, p.n_q_heads, 128))
        self._q_score = torch.Size((p.batch, p.n_idx_q_heads or p.n_q_heads, 128))
        self._s, self._i = torch.Size((p.batch, heads, p.max_len)), torch.Size((p.batch, heads, p.topk))
        self._rows = torch.Size((p.batch, heads, p.n_sink + p.topk + p.n_local, 128))
        self._type = B.element_type(p)
        self.status = torch.zeros((1,), dtype=torch.int32, device=self._dev)
        self.ws = torch.empty((max(B.skv_kv4_workspace_size(p), 16),), dtype=torch.uint8, device=self._dev)
        self.out = torch.empty(self._q, dtype=torch.bfloat16, device=self._dev)
        self.lse = torch.empty(self._q[:2], dtype=torch.float32, device=self._dev)
        self._st = self.status.data_ptr()
        self._outs = (self.out.data_ptr(), self.lse.data_ptr(), self.ws.data_ptr(), self.ws.numel(), self._st)
        self._score, self._attn = lib.skv_score_kv4, lib.skv_attn_kv4
        self._step, self._gather = lib.skv_decode_step_kv4, lib.skv_gather_kv4
        self._scores = self._idx = None

    def _new(self, shape, dtype, stream):
        """A tensor of the allocator's pool of the stream that writes it: the current stream's may hand out
        memory that work queued there has still to use."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            return torch.empty(shape, dtype=dtype, device=self._dev)

    def _own_scores(self, stream):
        if self._scores is None:
            self._scores = self._new(self._s, torch.float32, stream)
        return self._scores

    def _own_idx(self, stream):
        if self._idx is None:
            self._idx = self._new(self._i, torch.int32, stream)
        return self._idx

    @property
    def scores(self) -> torch.Tensor:
        """[batch, heads, max_len]; made when first used, for the stream of that use."""
        return self._own_scores(None)

    @property
    def idx(self) -> torch.Tensor:
        """[batch, heads, topk]; made when first used, for the stream of that use."""
        return self._own_idx(None)

    def _ptr(self, name, t, dtype, shape):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._device:
            raise ValueError(f"{name}: contiguous {dtype} {list(shape)} on {self._dev} expected")
        return B.list_ptr(self.p, t)

    def score(self, q_score, scores=None, stream=None):
        """Scores of the candidates into `scores` (the step's own unless given), which it returns."""
        scores = self._own_scores(stream) if scores is None else scores
        st = self._score(self._p, self._ptr("q_score", q_score, torch.bfloat16, self._q_score), self._pool, self._group,
                         self._ptr("scores", scores, torch.float32, self._s), self._st, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_score_kv4", st)
        return scores

    def topk(self, stream=None):
        """The selection of the step's own scores, into idx."""
        idx = self._own_idx(stream)
        if self.p.topk > 0:
            B.skv_topk(self.p, self._own_scores(stream), idx, self.ws, self.status, stream)
        return idx

    def _attend(self, q, idx, stream):
        st = self._attn(self._p, self._ptr("q", q, torch.bfloat16, self._q), self._pool, self._group,
                        None if idx is None else self._ptr("idx", idx, torch.int32, self._i), *self._outs,
                        B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_attn_kv4", st)
        return self.out, self.lse

    def attend(self, q, idx=None, stream=None):
        """(out, lse) over sink, selection (the step's own idx unless given) and window."""
        return self._attend(q, self._own_idx(stream) if idx is None else idx, stream)

    def attend_all(self, q, stream=None):
        """(out, lse) over every position of each history."""
        return self._attend(q, None, stream)

    def run(self, q, q_score=None, stream=None):
        """(out, lse) of one decode step; scores and idx hold its scores and selection."""
        st = self._step(self._p, self._ptr("q", q, torch.bfloat16, self._q),
                        None if q_score is None else self._ptr("q_score", q_score, torch.bfloat16, self._q_score),
                        self._pool, self._group, self._own_scores(stream).data_ptr(),
                        B.list_ptr(self.p, self._own_idx(stream)), *self._outs, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_decode_step_kv4", st)
        return self.out, self.lse

    def gather(self, idx=None, k_out=None, v_out=None, stream=None):
        """(k, v) [batch, heads, n_att, 128] of the problem's type: the attended rows' values; new tensors
        unless given.  Without a selection (topk 0) those of sink and window."""
        if idx is None and self.p.topk > 0:
            idx = self._own_idx(stream)
        ip = None if idx is None else self._ptr("idx", idx, torch.int32, self._i)
        k_out = self._new(self._rows, self._type, stream) if k_out is None else k_out
        v_out = self._new(self._rows, self._type, stream) if v_out is None else v_out
        st = self._gather(self._p, self._pool, self._group, ip, self._ptr("k_out", k_out, self._type, self._rows),
                          self._ptr("v_out", v_out, self._type, self._rows), self._st, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_gather_kv4", st)
        return k_out, v_out


class BlockTables:
    """Slot table, lengths and free blocks of a batch, kept on the GPU: `update(n_new, n_tokens)` is one
    skv_update_tables, whose positions and requests TokenStep.append() takes.  `free_blocks`: the
    stack's room, its first n_free entries (all, unless given) the free blocks, the last the first
    to be given.  The problem's seq_lens and the table are updated in place."""

    def __init__(self, problem: B.Problem, slot_table: torch.Tensor, free_blocks: torch.Tensor,
                 n_free: Optional[int] = None, base: int = 0):
        dev = problem.seq_lens.device
        n_free = free_blocks.numel() if n_free is None else n_free
        if not 0 <= n_free <= free_blocks.numel():
            raise ValueError("n_free: at most the stack's room")
        self.state = torch.tensor([n_free, 0, 0, 0], dtype=torch.int32).to(dev)
        self.p, self.tables = problem, B.Tables(slot_table, free_blocks, self.state, base)
        self.tables.check(problem)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._held = [*vars(problem).values(), *vars(self.tables).values()]
        self._dev, self._device, self._batch = dev, problem.seq_lens.get_device(), torch.Size((problem.batch,))
        self._none = tuple(torch.empty(0, dtype=t, device=dev) for t in (torch.int32, torch.int32, torch.int64))
        self._t, self._st = ctypes.byref(self.tables.c(problem)), self.status.data_ptr()
        self._call = B.lib().skv_update_tables

    @property
    def n_free(self) -> torch.Tensor:
        """Blocks on the stack, int32 [1] on the GPU."""
        return self.state[:1]

    def _new(self, n, stream):
        """Outputs, of the allocator's pool of the stream that writes them."""
        if n == 0:
            return self._none
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._new(n, None)
        return (torch.empty(n, dtype=torch.int32, device=self._dev), torch.empty(n, dtype=torch.int32, device=self._dev),
                torch.empty(n, dtype=torch.int64, device=self._dev))

    def update(self, n_new, n_tokens: int = 0, out=None, stream=None):
        """(positions, requests, slots) of the step's n_tokens rows: new tensors, unless given as `out`
        (slots may be None there)."""
        if n_new.dtype != torch.int32 or n_new.shape != self._batch or not n_new.is_contiguous() \
                or n_new.get_device() != self._device:
            raise ValueError(f"n_new: contiguous int32 {list(self._batch)} on {self._dev} expected")
        if out is None:
            rows = self._new(n_tokens, stream)
        else:
            rows = out
            for name, t, dtype in zip(("positions", "requests", "slots"), out, (torch.int32, torch.int32, torch.int64)):
                B.dense(self.p, name, t, dtype, (n_tokens,))
        at, req, slots = rows
        st = self._call(self._t, n_new.data_ptr(), n_tokens, at.data_ptr(), req.data_ptr(),
                        None if slots is None else slots.data_ptr(), self._st, B.raw_stream(self._device, stream))
        if st:
            raise B.SkvError("skv_update_tables", st)
        return rows
