// Scores, attention and the gather from a cache in 4 bits (cells: kv4.cuh).
//
//   score      <q, k^_t>,  k^ = s (c - 8) + z a group
//   attention  softmax(scale <q, k^_t>) over the history or a list, times v^_t
//
// Both walk tiles of 16 keys.  Keys are the rows and the query heads the columns of a
// product S^T = K Q^T (m16n8k16): with at most 16 heads a KV head this wastes nothing of the
// tensor core's 16 rows, and what it gives -- keys by heads -- is, transposed in registers
// (movmatrix), the second operand of O^T = V^T P^T.  Codes never become numbers in memory: a nibble
// masked out of its word is, as fp16, the subnormal c 2^-24 (from the low half of a byte) or
// c 2^-20 (from the high half), exactly, so an operand register of two codes costs one AND, and
// the powers of two go to the other operand (queries) or the result's rows (values).
//   logit   sum_g s_g (sum_j q_j c_j - 8 sum_j q_j) + sum_g z_g sum_{j in g} q_j
// The first product comes per group, scaled in fp32; what is left is a product of the words
// themselves -- a word is a pair of bf16 -- with the queries' group sums in three bf16 parts.
// Queries go to fp16 under a power of two of their own: bf16's 8 bits fit, and what falls under
// fp16's range is 2^-35 of the head's largest.
//   out     sum_t w_tg (c - 8) + sum_t p_t z_tg,  w_tg = p_t s_tg in fp16
// The maximum is a running one that moves only when a logit passes it by 2^7 (then everything
// is rescaled), and so is the power of two above the steps.
#include "attn_common.cuh"
#include "kv4.cuh"

namespace skv {
namespace {

constexpr int kW = 8;  // warps a CTA
constexpr int kMaxParts = 320;  // CTAs of an attention at most
constexpr int kSlotFloats = 16 * (kD + 2);  // a partial: O of 16 heads, then their (reference, sum)

struct Kv4Args {
  const __nv_bfloat16* q;
  PoolView pool;
  const int32_t* idx;
  const int32_t* seq_lens;
  int B, H, Hq, G, heads;  // H: rows of the kernel a request; heads: the pool's
  int max_len, ns, nl, k, bs;
  int cells, shift;        // of a block: its cells; log2 of its tokens, or -1
  unsigned n_gpu, n_host;  // blocks there (0 without a host pool)
  unsigned block_bytes;    // of a GPU block (of K, of V)
  int step_blocks, step_cells;  // kW tiles on
  int agg, Gi;             // scores
  float scale_log2;
  int32_t* status;
  float* scores;
  float* ws;      // partials [CTA][2][kSlotFloats], then desc
  int2* desc;     // [B * H]: the first CTA of a unit (bit 30: its second slot) and the last
  __nv_bfloat16* out;
  float* lse;
};

enum { kDense, kList, kScore };

// What a request of length L has to walk: tiles of 16 keys or list entries.
template <int MODE>
__device__ __forceinline__ int tiles_of(const Kv4Args& a, int L) {
  if (MODE == kDense) return (L + 15) >> 4;
  const Regions r = regions_of(L, a.ns, a.nl);
  if (MODE == kList) return (r.s_end + a.k + (L - r.l_start) + 15) >> 4;
  return r.l_start > r.s_end ? ((r.l_start + 15) >> 4) - (r.s_end >> 4) : 0;
}

__device__ __forceinline__ int len_of(const Kv4Args& a, int b) {
  const int L = __ldg(a.seq_lens + b);
  return L < 0 ? 0 : L > a.max_len ? a.max_len : L;
}

// A place in the walk: unit (b, h), tile of it; tiles are numbered b major, then h.
struct Cursor {
  int b, h, tile, nt, L;
};
template <int MODE>
__device__ __forceinline__ void settle(const Kv4Args& a, Cursor& c) {  // tile may lie past its unit
  while (c.tile >= c.nt) {
    c.tile -= c.nt;
    if (++c.h == a.H) {
      c.h = 0;
      do {
        if (++c.b >= a.B) return;
        c.L = len_of(a, c.b);
        c.nt = tiles_of<MODE>(a, c.L);
      } while (c.nt == 0);
    }
  }
}

// The CTAs' shares of T tiles: CTA c of n takes [T c / n, T (c + 1) / n).
__device__ __forceinline__ long long share(long long T, int n, int c) { return T * c / n; }
__device__ __forceinline__ int holder(long long T, int n, long long tile) { return (int)(((tile + 1) * n - 1) / T); }

// Every thread of the CTA gets the walk's length and the place where this CTA's share starts.
template <int MODE>
__device__ __forceinline__ void find_share(const Kv4Args& a, int min_tiles, long long* total, int* ctas,
                                           long long* t0, long long* t1, Cursor* c) {
  __shared__ long long s_warp[kW];
  __shared__ int s_at[3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.B + kW * 32 - 1) / (kW * 32), b0 = threadIdx.x * per, b1 = b0 + per < a.B ? b0 + per : a.B;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = blockIdx.x == 0 ? load_len(a.seq_lens, b, a.max_len, a.status) : len_of(a, b);
    mine += tiles_of<MODE>(a, L);
  }
  long long x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += u;
  }
  if (lane == 31) s_warp[warp] = x;
  if (threadIdx.x == 0) s_at[0] = -1;
  __syncthreads();
  long long before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w == warp) before = sum;
    sum += s_warp[w];
  }
  before += x - mine;
  const long long T = sum * a.H;
  long long n = (T + min_tiles - 1) / min_tiles;
  n = n < 1 ? 1 : n > gridDim.x ? gridDim.x : n;
  *total = T;
  *ctas = (int)n;
  *t0 = *t1 = 0;
  if (blockIdx.x < n) {
    *t0 = share(T, (int)n, blockIdx.x);
    *t1 = share(T, (int)n, blockIdx.x + 1);
  }
  if (*t1 > *t0 && before * a.H <= *t0 && *t0 < (before + mine) * a.H) {  // one thread's requests hold it
    long long at = *t0 - before * a.H;
    for (int b = b0; b < b1; ++b) {
      const int nt = tiles_of<MODE>(a, len_of(a, b));
      if (at < (long long)nt * a.H) {
        s_at[0] = b;
        s_at[1] = (int)(at / nt);
        s_at[2] = (int)(at % nt);
        break;
      }
      at -= (long long)nt * a.H;
    }
  }
  __syncthreads();
  c->b = s_at[0];
  if (c->b >= 0) {
    c->h = s_at[1];
    c->tile = s_at[2];
    c->L = len_of(a, c->b);
    c->nt = tiles_of<MODE>(a, c->L);
  }
}

// ---------------------------------------------------------------------------- a warp's ring
//
// A stage holds a tile as cells: K's codes and words, then V's.  V's rows of codes stand in
// another order and with their 16-byte chunks exchanged in pairs, so that the 8-byte loads of
// the second product meet no bank twice; the loads of K's rows are consecutive as they are.

__device__ __forceinline__ int v_place(int r) { return (r & 8) | ((r & 7) >> 1) | ((r & 1) << 2); }
__device__ __forceinline__ int v_chunk(int place, int c) { return c ^ (place & 2); }

template <int BYTES>
__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_cg16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The row of lane (lane & 15) on its way from its place in the walk to its address, a step an
// iteration, so that each step's load has a tile's time to arrive.
struct Row {
  int t;            // position, as found (a selected one unchecked); -1: none
  int e, block;     // its table entry, that one's index
  int b, h, L;
  bool listed;      // from the selection: to be checked
};

__device__ __forceinline__ void row_position(const Kv4Args& a, const Cursor& c, bool on, int r, Row& w) {
  w.b = c.b;
  w.h = c.h;
  w.L = c.L;
  w.t = -1;
  w.listed = false;
  if (!on) return;
  const int j = (c.tile << 4) + r;
  const Regions g = regions_of(c.L, a.ns, a.nl);
  if (j < g.s_end) {
    w.t = j;
  } else if (j < g.s_end + a.k) {
    w.t = __ldg(a.idx + ((size_t)c.b * a.H + c.h) * a.k + (j - g.s_end));
    w.listed = true;
  } else {
    const int t = g.l_start + (j - g.s_end - a.k);
    w.t = t < c.L ? t : -1;
  }
}

__device__ __forceinline__ void row_entry(const Kv4Args& a, bool reports, Row& w) {
  if (w.listed && w.t >= 0) {
    const Regions g = regions_of(w.L, a.ns, a.nl);
    if (w.t < g.s_end || w.t >= g.l_start) {
      if (reports) flag(a.status, SKV_DEV_BAD_INDEX);
      w.t = -1;
    }
  }
  w.e = 0;
  if (w.t >= 0) {
    w.block = a.shift >= 0 ? w.t >> a.shift : w.t / a.bs;
    w.e = __ldg(table_row(a.pool, w.b, a.pool.hdiv == 1 ? w.h : w.h / a.pool.hdiv, a.heads) + w.block);
  }
}

// The row's number in its pool, bit 31: the host's (pools have fewer than 2^31 rows).
constexpr uint32_t kNoRow = 0xffffffffu;
__device__ __forceinline__ uint32_t row_id(const Kv4Args& a, bool reports, const Row& w) {
  if (w.t < 0) return kNoRow;
  const uint32_t ph = a.pool.hdiv == 1 ? w.h : w.h / a.pool.hdiv, off = w.t - w.block * a.bs;
  if (w.e >= 0) {
    if ((uint32_t)w.e < a.n_gpu) return (a.pool.per_head ? w.e : w.e * a.heads + ph) * a.bs + off;
  } else if (~(uint32_t)w.e < a.n_host) {
    return ((~(uint32_t)w.e * a.heads + ph) * a.bs + off) | 0x80000000u;
  }
  if (reports) flag(a.status, SKV_DEV_BAD_SLOT);
  return kNoRow;
}

// Where a lane's 16-byte chunk of V's codes goes: chunk `lane` of the first eight rows (of the
// others 512 bytes on).
__device__ __forceinline__ uint32_t v_chunk_at(int lane) {
  const int p = v_place(lane >> 2);
  return p * kCodeBytes + v_chunk(p, lane & 3) * 16;
}

// Feeders: a warp issues its tiles' copies S - 1 tiles ahead of the one it computes, a commit
// group a tile.  issue() is called once a tile (before it is computed, and S - 1 times at
// the start); live() then tells which rows of the tile to be computed are there.

// Whole cells: a history's tiles.  The entry of a tile is loaded when the one before it is
// issued, so it has a tile's time to arrive.  What a unit's tiles share -- its table row, the
// pools at its head -- is found when the unit is entered, and a block's number and the
// cell in it move on without a division.
template <int MODE, int NG, bool V, int S>
struct CellFeeder {
  static constexpr int kStage = (V ? 2 : 1) * kv4_cell(NG);
  const Kv4Args& a;
  uint32_t to, end;  // the stage that is filled next, the ring's end
  uint32_t v_at;
  Cursor c;  // the tile that is issued next
  int left, e;
  int block, in;      // the tile's block, its cell there
  const int32_t* row;  // the unit's entries
  const unsigned char *k, *v;  // this lane's first chunk of the head's cells in GPU block 0
  uint32_t bad;  // of the tiles issued, the last in bit 0: no such block

  __device__ __forceinline__ CellFeeder(const Kv4Args& args, uint32_t ring, uint32_t*, Cursor at, int n)
      : a(args), to(ring), end(ring + S * kStage), v_at(v_chunk_at(threadIdx.x & 31)), c(at), left(n), bad(0) {
    if (left > 0) enter();
  }
  __device__ __forceinline__ void enter() {
    settle<MODE>(a, c);
    const int cell = (MODE == kScore ? regions_of(c.L, a.ns, a.nl).s_end >> 4 : 0) + c.tile;
    block = cell / a.cells;
    in = cell - block * a.cells;
    row = table_row(a.pool, c.b, c.h, a.heads);
    const size_t at = (a.pool.per_head ? 0 : (size_t)c.h * a.cells * kv4_cell(NG)) + (threadIdx.x & 31) * 16;
    k = (const unsigned char*)a.pool.gpu_k + at;
    v = (const unsigned char*)a.pool.gpu_v + at;
    e = __ldg(row + block);
  }
  __device__ __forceinline__ void copy(const unsigned char* ks, const unsigned char* vs) {
    const int lane = threadIdx.x & 31;
    const uint32_t dst = to + lane * 16;
    cp_async_cg16(dst, ks);
    cp_async_cg16(dst + 512, ks + 512);
    if (V) {
      cp_async_cg16(to + kv4_cell(NG) + v_at, vs);
      cp_async_cg16(to + kv4_cell(NG) + v_at + 512, vs + 512);
    }
    if (lane < 4 * NG) {
      cp_async_cg16(dst + 1024, ks + 1024);
      if (V) cp_async_cg16(dst + kv4_cell(NG) + 1024, vs + 1024);
    }
  }
  __device__ __forceinline__ void issue() {
    bad <<= 1;
    if (left > 0) {
      if ((unsigned)e < a.n_gpu) {
        const size_t at = (size_t)(unsigned)e * a.block_bytes + in * kv4_cell(NG);
        copy(k + at, v + at);
      } else if (e < 0 && ~(unsigned)e < a.n_host) {
        const size_t at = (((size_t)~(unsigned)e * a.heads + c.h) * a.cells + in) * kv4_cell(NG) + (threadIdx.x & 31) * 16;
        copy((const unsigned char*)a.pool.host_k + at, (const unsigned char*)a.pool.host_v + at);
      } else {
        if ((threadIdx.x & 31) == 0) flag(a.status, SKV_DEV_BAD_SLOT);
        bad |= 1u;
      }
      if (--left > 0) {
        c.tile += kW;
        if (c.tile >= c.nt) {
          enter();
        } else {
          block += a.step_blocks;
          in += a.step_cells;
          if (in >= a.cells) in -= a.cells, ++block;
          e = __ldg(row + block);
        }
      }
    }
    cp_async_commit();
    to = to + kStage == end ? end - S * kStage : to + kStage;
  }
  // tile `tile` of a request of L positions, S - 1 issues ago
  __device__ __forceinline__ uint32_t live(int L, int tile, int) const {
    if (bad >> (S - 1) & 1u) return 0u;
    const int n = L - (tile << 4);
    return n >= 16 ? 0xffffu : (1u << n) - 1u;
  }
};

// Single rows: a list's tiles.  Lanes 0 .. 15 (and 16 .. 31 with them) find a row each, a step an
// issue: its place's position, that one's entry, the row -- so each load has a tile's time to arrive.
template <int MODE, int NG, bool V, int S>
struct RowFeeder {
  static constexpr int kStage = 2 * kv4_cell(NG);
  const Kv4Args& a;
  uint32_t to, end, v_at;
  uint32_t* masks;
  Cursor c;  // the tile whose positions are found next
  int left, slot;
  Row r1, r0;  // position on its way; entry on its way

  __device__ __forceinline__ RowFeeder(const Kv4Args& args, uint32_t ring, uint32_t* masks_, Cursor at, int n)
      : a(args), to(ring), end(ring + S * kStage), v_at(v_chunk_at(threadIdx.x & 31)), masks(masks_), c(at), left(n),
        slot(0) {
    if (left > 0) settle<MODE>(a, c);
    position();
    advance();
  }
  __device__ __forceinline__ void position() {
    row_position(a, c, left > 0, threadIdx.x & 15, r1);
    if (--left > 0) {
      c.tile += kW;
      if (c.tile >= c.nt) settle<MODE>(a, c);
    }
  }
  __device__ __forceinline__ void advance() {
    r0 = r1;
    row_entry(a, (threadIdx.x & 31) < 16, r0);
    position();
  }
  __device__ __forceinline__ void issue() {
    const int lane = threadIdx.x & 31;
    const uint32_t row = row_id(a, lane < 16, r0);
    const uint32_t live = __ballot_sync(0xffffffffu, row != kNoRow) & 0xffffu;
    if (lane == 0) masks[slot] = live;
    auto at = [&](uint32_t r, bool v) {  // the row's cell
      const unsigned char* base = (const unsigned char*)(r >> 31 ? (v ? a.pool.host_v : a.pool.host_k)
                                                                 : (v ? a.pool.gpu_v : a.pool.gpu_k));
      return base + (size_t)(r >> 4 & 0x7ffffffu) * kv4_cell(NG);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t r = __shfl_sync(0xffffffffu, row, (lane >> 2) + 8 * i);
      if (r != kNoRow) {
        const int off = (int)(r & 15u) * kCodeBytes + (lane & 3) * 16;
        cp_async_cg16(to + lane * 16 + 512 * i, at(r, false) + off);
        cp_async_cg16(to + kv4_cell(NG) + v_at + 512 * i, at(r, true) + off);
      }
    }
    if (row != kNoRow) {
      const uint32_t dst = to + (lane >= 16 ? kv4_cell(NG) : 0) + 16 * kCodeBytes + (lane & 15) * 4 * NG;
      const unsigned char* src = at(row, lane >= 16) + 16 * kCodeBytes + (row & 15u) * 4 * NG;
      if (NG == 4)
        cp_async_cg16(dst, src);
      else
        cp_async_ca<4 * NG>(dst, src);
    }
    cp_async_commit();
    to = to + kStage == end ? end - S * kStage : to + kStage;
    slot = slot == S - 1 ? 0 : slot + 1;
    advance();
  }
  __device__ __forceinline__ uint32_t live(int, int, int stage) const { return masks[stage]; }
};

// ---------------------------------------------------------------------------- the products

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same of zero accumulators, which take no registers
__device__ __forceinline__ void mma_f16_new(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_new(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 u;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(addr));
  return u;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t u;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(addr));
  return u;
}
template <int NG>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if constexpr (NG == 4) {
    const uint4 u = lds128(addr);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = lds64(addr);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = lds32(addr);
  }
}
__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float centre_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The four operand registers of two bytes' worth of codes, in the order low and high half of
// the first byte, low and high half of the second: subnormal fp16 pairs, 2^-24 and 2^-20 a unit.
__device__ __forceinline__ void spread(uint32_t x, uint32_t* r) {
  const uint32_t y = x >> 8;
  r[0] = x & 0x000f000fu;
  r[1] = x & 0x00f000f0u;
  r[2] = y & 0x000f000fu;
  r[3] = y & 0x00f000f0u;
}

// A power of two that brings |x| <= mx under 2^10 (its own inverse is exact too).
__device__ __forceinline__ float fit(float mx) {
  int e = 263 - (int)((__float_as_uint(mx) >> 23) & 255u);
  e = e < 1 ? 1 : e > 254 ? 254 : e;
  return __uint_as_float((uint32_t)e << 23);
}

// Queries as the second operand: columns are heads, k-step j the entries 16 j .. 16 j + 15 in
// the order that the codes come in; wz: the group sums, three bf16 parts, against words.
template <int NT>
struct QFrag {
  uint32_t b[NT][8][2];
  uint32_t wz[NT][3];
  float unit[NT][2];  // what a logit of heads 2 t, 2 t + 1 comes in: 2^20 / their power of two
};

// the column's entries 16 j + 4 t .. + 3 for this lane are x[j][0..3], already under a power of
// two; a register's pairs are entries 0 and 2, 1 and 3
__device__ __forceinline__ void column(const float (&x)[8][4], uint32_t (&b)[8][2]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    b[j][0] = pack_f16(16.f * x[j][0], 16.f * x[j][2]);
    b[j][1] = pack_f16(x[j][1], x[j][3]);
  }
}
// what a word's halves meet: sums over the groups, of lane t the t-th group's
template <int NG>
__device__ __forceinline__ void column_sums(const float (&x)[8][4], uint32_t (&wz)[3], bool on) {
  const int t = threadIdx.x & 3;
  float part[NG], z = 0.f;
#pragma unroll
  for (int g = 0; g < NG; ++g) part[g] = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[j * NG / 8] += (x[j][0] + x[j][1]) + (x[j][2] + x[j][3]);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    part[g] += __shfl_xor_sync(0xffffffffu, part[g], 1);
    part[g] += __shfl_xor_sync(0xffffffffu, part[g], 2);
    if (g == t) z = part[g];
  }
  // in the products' unit
  z = on && t < NG ? z * 0x1p-20f : 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float h = __bfloat162float(__float2bfloat16_rn(z));
    wz[i] = tc::pack_bf16(-8.f * h, h);
    z -= h;
  }
}

// the largest |x| of a column (its four lanes hold all entries)
__device__ __forceinline__ float largest(const float (&x)[8][4]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(x[j][i]));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

__device__ __forceinline__ void load_q4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(u.x << 16);
  x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16);
  x[3] = __uint_as_float(u.y & 0xffff0000u);
}

// heads j0 .. j0 + n of a request's queries as columns
template <int NG, int NT>
__device__ __forceinline__ void load_heads(const __nv_bfloat16* q, int n, QFrag<NT>& f) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[8][4];
    const bool on = 8 * nt + g < n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = 0.f;
      if (on) load_q4(q + (size_t)(8 * nt + g) * kD + 16 * j + 4 * t, x[j]);
    }
    const float s = fit(largest(x));
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] *= s;
    column(x, f.b[nt]);
    column_sums<NG>(x, f.wz[nt], true);
    const float u = 0x1p20f / s;
    f.unit[nt][0] = __shfl_sync(0xffffffffu, u, 8 * t);
    f.unit[nt][1] = __shfl_sync(0xffffffffu, u, 8 * t + 4);
  }
}

// the mean of n heads in three fp16 parts, columns 0, 1 and 2
template <int NG>
__device__ __forceinline__ void load_mean(const __nv_bfloat16* q, int n, QFrag<1>& f) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float x[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] = 0.f;
  for (int h = 0; h < n; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float y[4];
      load_q4(q + (size_t)h * kD + 16 * j + 4 * t, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] += y[i];
    }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] /= (float)n;
  const float s = fit(largest(x));
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j][i] *= s;
  column_sums<NG>(x, f.wz[0], g == 0);
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y = x[j][i], part = 0.f;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const float h = __half2float(__float2half_rn(y));
        if (k == g) part = h;
        y -= h;
      }
      x[j][i] = part;
    }
  column(x, f.b[0]);
  f.unit[0][0] = f.unit[0][1] = 0x1p20f / s;
}

// The logits of a tile, in the columns' units: c[nt][0..1] key g of heads 2 t, 2 t + 1; [2..3] key g + 8.
// A row's logits depend on that row alone: those of rows that are not there are anything.
template <int NG, int NT>
__device__ __forceinline__ void logits(uint32_t stage, const QFrag<NT>& f, float (&c)[NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint4 k0 = lds128(stage + g * kCodeBytes + t * 16), k1 = lds128(stage + (g + 8) * kCodeBytes + t * 16);
  const uint32_t words = stage + 16 * kCodeBytes;
  uint32_t w0[NG], w1[NG];
  lds_words<NG>(words + g * 4 * NG, w0);
  lds_words<NG>(words + (g + 8) * 4 * NG, w1);
  uint32_t aw[4];
  aw[0] = t < NG ? lds32(words + (g * NG + t) * 4) : 0u;
  aw[1] = t < NG ? lds32(words + ((g + 8) * NG + t) * 4) : 0u;
  aw[2] = aw[0];
  aw[3] = aw[1];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    mma_bf16_new(c[nt], aw, f.wz[nt][0], f.wz[nt][1]);
    tc::mma_bf16(c[nt], aw, f.wz[nt][2], 0u);
  }
  float acc[NT][4];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {  // two k-steps: bytes 2 jj, 2 jj + 1 of the lane's two runs of eight
    const uint32_t sel = jj & 1 ? 0x7632u : 0x5410u;
    uint32_t r0[4], r1[4];
    spread(__byte_perm(jj < 2 ? k0.x : k0.y, jj < 2 ? k0.z : k0.w, sel), r0);
    spread(__byte_perm(jj < 2 ? k1.x : k1.y, jj < 2 ? k1.z : k1.w, sel), r1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 2 * jj + i;
      const uint32_t ar[4] = {r0[2 * i], r1[2 * i], r0[2 * i + 1], r1[2 * i + 1]};
      constexpr int kSteps = 8 / NG;  // of a group
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (j % kSteps == 0)
          mma_f16_new(acc[nt], ar, f.b[nt][j][0], f.b[nt][j][1]);
        else
          mma_f16(acc[nt], ar, f.b[nt][j][0], f.b[nt][j][1]);
        if (j % kSteps == kSteps - 1) {
          const float s0 = step_of(w0[j / kSteps]), s1 = step_of(w1[j / kSteps]);
          c[nt][0] = fmaf(s0, acc[nt][0], c[nt][0]);
          c[nt][1] = fmaf(s0, acc[nt][1], c[nt][1]);
          c[nt][2] = fmaf(s1, acc[nt][2], c[nt][2]);
          c[nt][3] = fmaf(s1, acc[nt][3], c[nt][3]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- attention

// A warp's state of a unit: p_t = 2^(x_t - r), r = the running maximum + the steps' power - 7.
template <int NG, int NT>
struct State {
  float m[NT][2], l[NT][2];
  float ref[NT][2], top[NT][2];  // -r; the logit in its column's unit past which the maximum moves
  float o[NT][8][4];  // rows 2 g (2^-24 a unit) and 2 g + 1 (2^-20) of entries 16 i, columns heads 2 t, 2 t + 1
  float z[NT][NG][2];
  int sigma;          // steps are below 2^(sigma + 1)
};
constexpr float kFloor = -3.0e38f;
constexpr int kSigmaMin = -60, kSigmaMax = 120;

template <int NG, int NT>
__device__ __forceinline__ void clear(State<NG, NT>& s) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.m[nt][i] = kFloor;
      s.ref[nt][i] = -kFloor;
      s.top[nt][i] = kFloor;
      s.l[nt][i] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) s.z[nt][g][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.o[nt][i][j] = 0.f;
  }
  s.sigma = kSigmaMin;
}

// A maximum or a power of the steps that a tile has passed: everything in the new reference.
template <int NG, int NT>
__device__ __forceinline__ void rescale(State<NG, NT>& s, const float (&c)[NT][4], const float (&kf)[NT][2],
                                        float smax) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, off));
  int e = (int)((__float_as_uint(smax) >> 23) & 255u) - 127;
  e = e > kSigmaMax ? kSigmaMax : e;
  const int sigma = e > s.sigma ? e : s.sigma;
  const float ds = (float)(s.sigma - sigma);
  s.sigma = sigma;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float m = fmaxf(c[nt][i], c[nt][i + 2]) * kf[nt][i];
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      m = fmaxf(m, s.m[nt][i]);
      f[i] = ex2(s.m[nt][i] - m + ds);
      s.m[nt][i] = m;
      s.ref[nt][i] = 7.f - (float)sigma - m;
      s.top[nt][i] = (m + 7.f) / kf[nt][i];
      s.l[nt][i] *= f[i];
#pragma unroll
      for (int g = 0; g < NG; ++g) s.z[nt][g][i] *= f[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.o[nt][i][j] *= f[j & 1];
  }
}

template <int NG, int NT>
__device__ __forceinline__ void attend_tile(uint32_t stage, uint32_t mask, const QFrag<NT>& f, const float (&kf)[NT][2],
                                            State<NG, NT>& s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float c[NT][4];
  logits<NG, NT>(stage, f, c);
  const uint32_t vc = stage + kv4_cell(NG), words = vc + 16 * kCodeBytes;
  uint32_t w0[NG], w1[NG];
  lds_words<NG>(words + g * 4 * NG, w0);
  lds_words<NG>(words + (g + 8) * 4 * NG, w1);
  const bool on0 = mask >> g & 1u, on1 = mask >> (g + 8) & 1u;
  if (mask != 0xffffu) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      w0[i] = on0 ? w0[i] : 0u;
      w1[i] = on1 ? w1[i] : 0u;
    }
  }
  // (each lane of a quad looks at a group's step)
  const uint32_t mine = words + (t & (NG - 1)) * 4;
  const float smax = fmaxf(on0 ? fabsf(step_of(lds32(mine + g * 4 * NG))) : 0.f,
                           on1 ? fabsf(step_of(lds32(mine + (g + 8) * 4 * NG))) : 0.f);
  bool past = smax >= __uint_as_float((uint32_t)(s.sigma + 128) << 23);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (mask != 0xffffu && !(i < 2 ? on0 : on1)) c[nt][i] = -INFINITY;
      past |= c[nt][i] > s.top[nt][i & 1];
    }
  if (__any_sync(0xffffffffu, past)) rescale<NG, NT>(s, c, kf, smax);
  // Every other key's codes come as 15 - c and its weights negative: w c - w' (15 - c') + 15 w'.  Codes
  // are 7.5 on average, and a long sum of them on one side of zero would lose to the tensor core's
  // truncation what the centring takes off again (a million keys: 1 % of the output).  With the
  // codes' own 8, the even keys' stand 8 too high and the odd ones' 7 too low.
  const float off = g & 1 ? 7.f : -8.f, sign = g & 1 ? -1.f : 1.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[nt][i] = ex2(fmaf(c[nt][i], kf[nt][i & 1], s.ref[nt][i & 1]));
    s.l[nt][0] += c[nt][0] + c[nt][2];
    s.l[nt][1] += c[nt][1] + c[nt][3];
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const float y0 = fmaf(off, step_of(w0[i]), centre_of(w0[i])), y1 = fmaf(off, step_of(w1[i]), centre_of(w1[i]));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s.z[nt][i][0] = fmaf(c[nt][0], y0, fmaf(c[nt][2], y1, s.z[nt][i][0]));
      s.z[nt][i][1] = fmaf(c[nt][1], y0, fmaf(c[nt][3], y1, s.z[nt][i][1]));
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[nt][i] *= sign;
  // the second product: weights times steps, transposed, a group at a time
  uint2 v[4];
  {
    const uint32_t row = vc + t * kCodeBytes + (v_chunk(t, g >> 1) << 4) + ((g & 1) << 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds64(row + i * 4 * kCodeBytes);  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
    v[1] = make_uint2(~v[1].x, ~v[1].y);
    v[3] = make_uint2(~v[3].x, ~v[3].y);
  }
  uint32_t wb[NT][2];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    const uint32_t sel = jj & 1 ? 0x7632u : 0x5410u;
    uint32_t r0[4], r1[4];
    spread(__byte_perm(jj < 2 ? v[0].x : v[0].y, jj < 2 ? v[1].x : v[1].y, sel), r0);
    spread(__byte_perm(jj < 2 ? v[2].x : v[2].y, jj < 2 ? v[3].x : v[3].y, sel), r1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 2 * jj + i;
      constexpr int kSteps = 8 / NG;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (j % kSteps == 0) {
          const float s0 = step_of(w0[j / kSteps]), s1 = step_of(w1[j / kSteps]);
          wb[nt][0] = tc::movmatrix_t(pack_f16(c[nt][0] * s0, c[nt][1] * s0));
          wb[nt][1] = tc::movmatrix_t(pack_f16(c[nt][2] * s1, c[nt][3] * s1));
        }
        const uint32_t ar[4] = {r0[2 * i], r0[2 * i + 1], r1[2 * i], r1[2 * i + 1]};
        mma_f16(s.o[nt][j], ar, wb[nt][0], wb[nt][1]);
      }
    }
  }
}

template <int NG, int NT>
struct AttnShape {
  // Stages and CTAs a SM: one column tile, 16 warps with two tiles of 2.5 KB ahead of them each;
  // two column tiles take the registers of two CTAs, and one stage more.
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kCtas = NT == 1 ? 2 : 1;
  static constexpr int kRing = kW * kStages * 2 * kv4_cell(NG);
  static constexpr int kRow = kD + 4;  // floats of a head's partial row: heads 2 t, 2 t + 2 an eighth of the banks apart
  static constexpr int kOut = kW * 8 * NT * kRow * 4;
  static constexpr int kSmem = kRing + kOut;
};

template <int MODE, int NG, int S>
struct Pick {
  using type = CellFeeder<MODE, NG, true, S>;
};
template <int NG, int S>
struct Pick<kList, NG, S> {
  using type = RowFeeder<kList, NG, true, S>;
};

template <int NG, int NT, int MODE>
__global__ void __launch_bounds__(32 * kW, AttnShape<NG, NT>::kCtas) kv4_attn_kernel(const Kv4Args a) {
  using Shape = AttnShape<NG, NT>;
  constexpr int S = Shape::kStages, HC = 8 * NT;  // columns
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t s_mask[MODE == kList ? kW : 1][S];
  __shared__ float2 s_ml[kW][HC], s_tot[HC];
  __shared__ float s_f[HC][kW];
  float* s_o = reinterpret_cast<float*>(smem + Shape::kRing);
  pdl_release();
  pdl_wait();
  long long T, t0, t1;
  int n;
  Cursor u;
  find_share<MODE>(a, kW, &T, &n, &t0, &t1, &u);
  if (t1 <= t0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mine = t1 - t0 > warp ? (int)((t1 - t0 - warp + kW - 1) / kW) : 0;
  Cursor at = u;
  at.tile += warp;
  constexpr uint32_t kStage = 2 * kv4_cell(NG);
  const uint32_t ring = smem_u32(smem) + warp * S * kStage;
  typename Pick<MODE, NG, S>::type feed(a, ring, s_mask[MODE == kList ? warp : 0], at, mine);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) feed.issue();
  int next = warp, seg = 0, stage = 0;  // next: this warp's next tile of the share
  for (long long f = t0; f < t1; ++seg) {
    const long long first = f - u.tile, end = first + u.nt < t1 ? first + u.nt : t1;
    QFrag<NT> q;
    load_heads<NG, NT>(a.q + ((size_t)u.b * a.Hq + (size_t)u.h * a.G) * kD, a.G, q);
    float kf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) kf[nt][0] = q.unit[nt][0] * a.scale_log2, kf[nt][1] = q.unit[nt][1] * a.scale_log2;
    State<NG, NT> s;
    clear(s);
    const int last = (int)(end - t0), base = (int)(first - t0);  // (a share has fewer tiles than 2^31)
    for (; next < last; next += kW) {
      cp_async_wait<S - 2>();
      __syncwarp();
      feed.issue();  // into the stage of the tile before this one
      const uint32_t mask = feed.live(u.L, next - base, stage);
      if (mask != 0u) attend_tile<NG, NT>(ring + stage * kStage, mask, q, kf, s);
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    // the warp's sums, then the CTA's
    float* row = s_o + warp * HC * Shape::kRow;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = 8 * nt + 2 * t + i;
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
          s.l[nt][i] += __shfl_xor_sync(0xffffffffu, s.l[nt][i], off);
#pragma unroll
          for (int k = 0; k < NG; ++k) s.z[nt][k][i] += __shfl_xor_sync(0xffffffffu, s.z[nt][k][i], off);
        }
        if (g == 0) s_ml[warp][head] = make_float2(s.m[nt][i] + ((float)s.sigma - 7.f), s.l[nt][i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = s.z[nt][j * NG / 8][i];
          *reinterpret_cast<float2*>(row + head * Shape::kRow + 16 * j + 2 * g) =
              make_float2(fmaf(s.o[nt][j][i], 0x1p24f, z), fmaf(s.o[nt][j][i + 2], 0x1p20f, z));
        }
      }
    __syncthreads();
    if (threadIdx.x < HC * kW) {
      const int head = threadIdx.x >> 3, w = threadIdx.x & 7;
      const float2 v = s_ml[w][head];
      float m = v.x;
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      const float fw = ex2(v.x - m);
      float l = fw * v.y;
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      s_f[head][w] = fw;
      if (w == 0) s_tot[head] = make_float2(m, l);
    }
    __syncthreads();
    const bool whole = first >= t0 && first + u.nt <= t1;
    const size_t hq = (size_t)u.b * a.Hq + (size_t)u.h * a.G;
    float* slot = a.ws + ((size_t)blockIdx.x * 2 + (seg > 0)) * kSlotFloats;
    const int d = threadIdx.x & (kD - 1);
    for (int head = threadIdx.x / kD; head < a.G; head += 32 * kW / kD) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) o = fmaf(s_f[head][w], s_o[(w * HC + head) * Shape::kRow + d], o);
      const float2 tot = s_tot[head];
      if (whole) {
        a.out[(hq + head) * kD + d] = __float2bfloat16_rn(tot.y == 0.f ? 0.f : o / tot.y);
        if (d == 0 && a.lse) a.lse[hq + head] = tot.y == 0.f ? -INFINITY : kLn2 * (tot.x + log2f(tot.y));
      } else {
        slot[head * kD + d] = o;
        if (d == 0) *reinterpret_cast<float2*>(slot + 16 * kD + 2 * head) = tot;
      }
    }
    if (threadIdx.x == 0 && first >= t0)
      a.desc[(size_t)u.b * a.H + u.h] = make_int2((int)blockIdx.x | (seg > 0 ? 1 << 30 : 0), holder(T, n, first + u.nt - 1));
    __syncthreads();
    f = end;
    if (f < t1) {
      u.tile = u.nt;
      settle<MODE>(a, u);
    }
  }
  cp_async_wait<0>();
}

// The units that no CTA held alone: their partials joined, a CTA a head; the empty ones: zeros.
template <int MODE>
__global__ void __launch_bounds__(kD) kv4_merge_kernel(const Kv4Args a) {
  __shared__ float s_f[kMaxParts];
  __shared__ float s_red[2][kD / 32];
  pdl_release();
  pdl_wait();
  const long long unit = blockIdx.x / a.G;
  const int head = blockIdx.x - (int)unit * a.G, b = (int)(unit / a.H), h = (int)(unit - (long long)b * a.H);
  const int d = threadIdx.x, lane = d & 31, warp = d >> 5;
  const size_t hq = (size_t)b * a.Hq + (size_t)h * a.G + head;
  if (tiles_of<MODE>(a, len_of(a, b)) == 0) {
    a.out[hq * kD + d] = __float2bfloat16_rn(0.f);
    if (d == 0 && a.lse) a.lse[hq] = -INFINITY;
    return;
  }
  const int2 span = a.desc[unit];
  const int c0 = span.x & ((1 << 30) - 1), parts = span.y - c0 + 1;
  if (parts == 1) return;
  const float* slots = a.ws + (size_t)c0 * 2 * kSlotFloats;
  const size_t first = span.x >> 30 ? kSlotFloats : 0;  // the others begin with this unit
  auto slot = [&](int i) { return slots + (i == 0 ? first : (size_t)i * 2 * kSlotFloats); };
  float m = kFloor;
  for (int i = d; i < parts; i += kD) m = fmaxf(m, slot(i)[16 * kD + 2 * head]);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) s_red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kD / 32; ++w) m = fmaxf(m, s_red[0][w]);
  float l = 0.f;
  for (int i = d; i < parts; i += kD) {
    const float2 v = *reinterpret_cast<const float2*>(slot(i) + 16 * kD + 2 * head);
    const float f = ex2(v.x - m);
    s_f[i] = f;
    l = fmaf(f, v.y, l);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if (lane == 0) s_red[1][warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kD / 32; ++w) l += s_red[1][w];
  float o = 0.f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) o = fmaf(s_f[i], slot(i)[head * kD + d], o);
  a.out[hq * kD + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  if (d == 0 && a.lse) a.lse[hq] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

// ---------------------------------------------------------------------------- scores

constexpr int kScoreStages = 4;

template <int NG, int NT, int AGG>
__global__ void __launch_bounds__(32 * kW, 2) kv4_score_kernel(const Kv4Args a) {
  constexpr int S = kScoreStages;
  extern __shared__ __align__(128) unsigned char smem[];
  pdl_release();
  pdl_wait();
  long long T, t0, t1;
  int n;
  Cursor u;
  find_share<kScore>(a, kW, &T, &n, &t0, &t1, &u);
  if (t1 <= t0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int mine = t1 - t0 > warp ? (int)((t1 - t0 - warp + kW - 1) / kW) : 0;
  Cursor at = u;
  at.tile += warp;
  const uint32_t ring = smem_u32(smem) + warp * S * kv4_cell(NG);
  CellFeeder<kScore, NG, false, S> feed(a, ring, nullptr, at, mine);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) feed.issue();
  int next = warp, stage = 0;
  for (long long f = t0; f < t1;) {
    const long long first = f - u.tile, end = first + u.nt < t1 ? first + u.nt : t1;
    const int last = (int)(end - t0);
    if (next < last) {
      QFrag<NT> q;
      const __nv_bfloat16* qp = a.q + ((size_t)u.b * a.H + u.h) * a.Gi * kD;
      if constexpr (AGG == SKV_AGG_MEAN)
        load_mean<NG>(qp, a.Gi, q);
      else
        load_heads<NG, NT>(qp, a.Gi, q);
      const Regions rg = regions_of(u.L, a.ns, a.nl);
      const int rows = AGG == SKV_AGG_HEAD ? a.Gi : 1;  // score rows of the unit
      float* out = a.scores + ((size_t)u.b * a.H + u.h) * rows * a.max_len;
      int k0 = (rg.s_end & ~15) + (next - (int)(first - t0)) * 16 + g;
      for (; next < last; next += kW, k0 += 16 * kW) {
        cp_async_wait<S - 2>();
        __syncwarp();
        feed.issue();
        const bool there = !(feed.bad >> (S - 1) & 1u);
        float c[NT][4];
        logits<NG, NT>(ring + stage * kv4_cell(NG), q, c);
        stage = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // keys g, g + 8
          const int key = k0 + 8 * i;
          const bool in = key >= rg.s_end && key < rg.l_start;
          if constexpr (AGG == SKV_AGG_HEAD) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int head = 8 * nt + 2 * t + j;
                if (in && head < a.Gi)
                  out[(size_t)head * a.max_len + key] = there ? c[nt][2 * i + j] * q.unit[nt][j] : NAN;
              }
          } else {
            float v;
            if constexpr (AGG == SKV_AGG_MAX) {
              v = -INFINITY;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float x = c[nt][2 * i + j] * q.unit[nt][j];
                  if (8 * nt + 2 * t + j < a.Gi) v = max_nan(v, x);
                }
              v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
              v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
            } else {  // columns 0, 1 here, 2 in the next lane
              v = (__shfl_down_sync(0xffffffffu, c[0][2 * i], 1) + c[0][2 * i + 1] + c[0][2 * i]) * q.unit[0][0];
            }
            if (t == 0 && in) out[key] = there ? v : NAN;
          }
        }
      }
    }
    f = end;
    if (f < t1) {
      u.tile = u.nt;
      settle<kScore>(a, u);
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------- gather

// Four lanes a row: 16 bytes of codes each, four consecutive entries of every 16.
template <int NG, typename T>
__global__ void __launch_bounds__(256) kv4_gather_kernel(const Kv4Args a, T* k_out, T* v_out, int n_att) {
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = lane & 3;
  const long long rows = (long long)a.B * a.H * n_att, warps = (long long)gridDim.x * 8;
  for (long long r = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 8 + (lane >> 2); r < rows; r += warps * 8) {
    const long long unit = r / n_att;
    const int j = (int)(r - unit * n_att);
    Cursor c;
    c.b = (int)(unit / a.H);
    c.h = (int)(unit - (long long)c.b * a.H);
    c.tile = j >> 4;
    c.L = t == 0 && j == 0 && c.h == 0 ? load_len(a.seq_lens, c.b, a.max_len, a.status) : len_of(a, c.b);
    c.nt = 0;
    Row w;
    row_position(a, c, true, j & 15, w);
    row_entry(a, t == 0, w);
    const uint32_t at = row_id(a, t == 0, w);
    const bool host = at >> 31;
    const size_t cell = (size_t)(at >> 4 & 0x7ffffffu) * kv4_cell(NG);
    const int rc = (int)(at & 15u);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      T* out = kv ? v_out : k_out;
      if (out == nullptr) continue;
      const unsigned char* src =
          (const unsigned char*)(kv ? (host ? a.pool.host_v : a.pool.gpu_v) : (host ? a.pool.host_k : a.pool.gpu_k));
      uint4 u = make_uint4(0, 0, 0, 0);
      float s[NG], z[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) s[i] = z[i] = 0.f;
      if (at != kNoRow) {
        u = __ldg(reinterpret_cast<const uint4*>(src + cell + rc * kCodeBytes) + t);
        const uint32_t* words = reinterpret_cast<const uint32_t*>(src + cell + 16 * kCodeBytes) + rc * NG;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const uint32_t x = __ldg(words + i);
          s[i] = step_of(x);
          z[i] = centre_of(x);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b0 = (i < 4 ? u.x : u.y) >> (8 * (i & 3)), b1 = (i < 4 ? u.z : u.w) >> (8 * (i & 3));
        const float si = s[i * NG / 8], zi = z[i * NG / 8];
        const float x[4] = {fmaf(si, (float)(int)(b0 & 15u) - 8.f, zi), fmaf(si, (float)(int)(b0 >> 4 & 15u) - 8.f, zi),
                            fmaf(si, (float)(int)(b1 & 15u) - 8.f, zi), fmaf(si, (float)(int)(b1 >> 4 & 15u) - 8.f, zi)};
        T* to = out + (size_t)r * kD + 16 * i + 4 * t;
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
        else
          *reinterpret_cast<uint2*>(to) = make_uint2(tc::pack_bf16(x[0], x[1]), tc::pack_bf16(x[2], x[3]));
      }
    }
  }
}

// ---------------------------------------------------------------------------- host

Kv4Args kv4_args(const skv_problem& p, const void* q, const PoolView& pool, int group, const int32_t* idx,
                 int32_t* status) {
  Kv4Args a = {};
  a.q = (const __nv_bfloat16*)q;
  a.pool = pool;
  if (a.pool.hdiv < 1) a.pool.hdiv = 1;
  a.idx = idx;
  a.seq_lens = p.seq_lens;
  a.B = p.batch;
  a.H = p.n_kv_heads;
  a.Hq = p.n_q_heads;
  a.G = p.n_q_heads / p.n_kv_heads;
  a.heads = a.H / a.pool.hdiv;
  a.max_len = p.max_len;
  a.ns = p.n_sink;
  a.nl = p.n_local;
  a.k = p.topk;
  a.bs = p.block_size;
  a.cells = p.block_size / kCellTokens;
  a.shift = -1;
  for (int i = 4; i < 31; ++i)
    if (p.block_size == 1 << i) a.shift = i;
  a.step_blocks = kW / a.cells;
  a.step_cells = kW % a.cells;
  a.block_bytes = (unsigned)((pool.per_head ? 1 : a.heads) * a.cells * kv4_cell(kD / group));
  a.n_gpu = (unsigned)pool.n_gpu;
  a.n_host = pool.host_k != nullptr ? (unsigned)pool.n_host : 0u;
  a.agg = p.group_agg;
  a.Gi = p.n_idx_q_heads / p.n_kv_heads;
  a.scale_log2 = (p.sm_scale > 0.f ? p.sm_scale : 1.f / sqrtf((float)p.d_qk)) * kLog2e;
  a.status = status;
  return a;
}

// CTAs for at most `tiles` tiles: all that are resident at once, a tile a warp at least
unsigned grid_of(long long tiles, int ctas) {
  long long n = (tiles + kW - 1) / kW, most = (long long)num_sms() * ctas;
  if (most > kMaxParts) most = kMaxParts;
  n = n < most ? n : most;
  return (unsigned)(n < 1 ? 1 : n);
}

template <int NG, int NT, int MODE>
skv_status launch_attn(const Kv4Args& a, long long tiles, cudaStream_t st) {
  using Shape = AttnShape<NG, NT>;
  const auto kernel = kv4_attn_kernel<NG, NT, MODE>;
  const skv_status prep = prepare_kernel((const void*)kernel, Shape::kSmem);
  if (prep != SKV_OK) return prep;
  if (launch_dependent(kernel, dim3(grid_of(tiles, Shape::kCtas)), dim3(32 * kW), Shape::kSmem, st, 1, a) !=
      cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  if (launch_dependent(kv4_merge_kernel<MODE>, dim3((unsigned)((long long)a.B * a.H * a.G)), dim3(kD), 0, st, 1, a) !=
      cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

template <int NG, int AGG>
skv_status launch_scores(const Kv4Args& a, long long tiles, cudaStream_t st) {
  const bool wide = AGG != SKV_AGG_MEAN && a.Gi > 8;
  const auto kernel = kv4_score_kernel<NG, 1, AGG>;
  const auto kernel2 = kv4_score_kernel<NG, AGG == SKV_AGG_MEAN ? 1 : 2, AGG>;
  constexpr int kSmem = kW * kScoreStages * kv4_cell(NG);
  const skv_status prep = prepare_kernel((const void*)(wide ? kernel2 : kernel), kSmem);
  if (prep != SKV_OK) return prep;
  if (launch_dependent(wide ? kernel2 : kernel, dim3(grid_of(tiles, 2)), dim3(32 * kW), kSmem, st, 1, a) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

template <int NG, typename T>
skv_status launch_gather4(const Kv4Args& a, void* k_out, void* v_out, int n_att, cudaStream_t st) {
  const long long warps = ((long long)a.B * a.H * n_att + 7) / 8, most = 8LL * num_sms();
  long long ctas = (warps + 7) / 8;
  if (ctas > most) ctas = most;
  if (launch_dependent(kv4_gather_kernel<NG, T>, dim3((unsigned)ctas), dim3(256), 0, st, 1, a, (T*)k_out, (T*)v_out,
                       n_att) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

size_t parts_bytes() { return align256((size_t)kMaxParts * 2 * kSlotFloats * 4); }

}  // namespace

size_t kv4_attn_workspace_bytes(const skv_problem& p) {
  return parts_bytes() + align256((size_t)p.batch * p.n_kv_heads * sizeof(int2));
}

skv_status launch_kv4_attn(const skv_problem& p, const void* q, const PoolView& pool, int group, const int32_t* idx,
                           void* out, float* lse, void* ws, int32_t* status, cudaStream_t st) {
  Kv4Args a = kv4_args(p, q, pool, group, idx, status);
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.ws = (float*)ws;
  a.desc = reinterpret_cast<int2*>((unsigned char*)ws + parts_bytes());
  const bool list = idx != nullptr;
  const long long n = list ? (long long)p.n_sink + p.topk + p.n_local : p.max_len;
  const long long tiles = (long long)a.B * a.H * ((n + 15) / 16);
#define KV4_ATTN(NG)                                                                                            \
  (a.G > 8 ? (list ? launch_attn<NG, 2, kList>(a, tiles, st) : launch_attn<NG, 2, kDense>(a, tiles, st))        \
           : (list ? launch_attn<NG, 1, kList>(a, tiles, st) : launch_attn<NG, 1, kDense>(a, tiles, st)))
  return group == 32 ? KV4_ATTN(4) : group == 64 ? KV4_ATTN(2) : KV4_ATTN(1);
#undef KV4_ATTN
}

skv_status launch_kv4_score(const skv_problem& p, const void* q, const PoolView& pool, int group, float* scores,
                            int32_t* status, cudaStream_t st) {
  Kv4Args a = kv4_args(p, q, pool, group, nullptr, status);
  a.scores = scores;
  const long long tiles = (long long)a.B * a.H * (((long long)p.max_len + 15) / 16 + 1);
#define KV4_SCORE(NG)                                                                 \
  (p.group_agg == SKV_AGG_MEAN  ? launch_scores<NG, SKV_AGG_MEAN>(a, tiles, st)       \
   : p.group_agg == SKV_AGG_MAX ? launch_scores<NG, SKV_AGG_MAX>(a, tiles, st)        \
                                : launch_scores<NG, SKV_AGG_HEAD>(a, tiles, st))
  return group == 32 ? KV4_SCORE(4) : group == 64 ? KV4_SCORE(2) : KV4_SCORE(1);
#undef KV4_SCORE
}

skv_status launch_kv4_gather(const skv_problem& p, const PoolView& pool, int group, const int32_t* idx, void* k_out,
                             void* v_out, int32_t* status, cudaStream_t st) {
  const Kv4Args a = kv4_args(p, nullptr, pool, group, idx, status);
  const int n_att = p.n_sink + p.topk + p.n_local;
  if (n_att == 0) return SKV_OK;
  const bool f32 = p.dtype == SKV_DTYPE_F32;
#define KV4_GATHER(NG)                                              \
  (f32 ? launch_gather4<NG, float>(a, k_out, v_out, n_att, st)      \
       : launch_gather4<NG, __nv_bfloat16>(a, k_out, v_out, n_att, st))
  return group == 32 ? KV4_GATHER(4) : group == 64 ? KV4_GATHER(2) : KV4_GATHER(1);
#undef KV4_GATHER
}

}  // namespace skv
