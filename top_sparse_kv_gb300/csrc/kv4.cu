// Scores, attention and the gather from a cache in 4 bits (cells: kv4.cuh).
//
//   score      <q, k^_t>,  k^ = s (c - 8) + z a group
//   attention  softmax(scale <q, k^_t>) over the history or a list, times v^_t
//
// Both walk tiles of 16 keys, a cell.  Keys are the rows and the query heads the columns of a
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
// The maximum is a running one that moves only when a logit passes it by 2^7 (then the head's sums
// are rescaled); w comes under a power of two that follows the largest of its head and group.
#include "attn_common.cuh"
#include "kv4.cuh"

namespace skv {
namespace {

constexpr int kMaxParts = 512;  // CTAs at most
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
  unsigned block_cells;    // of a GPU block
  int Gi;                  // scores: heads a KV head
  float scale_log2;
  int32_t* status;
  float* scores;
  float* ws;      // partials [CTA][2][kSlotFloats], then desc
  int2* desc;     // [B * H]: the first CTA of a unit (bit 30: its second slot) and the last
  __nv_bfloat16* out;
  float* lse;
};

enum { kDense, kList, kScore };

// What a request of length L has to walk: tiles of 16 keys, or of 16 list entries (scores: from the
// candidates' first cell on).
template <int MODE>
__device__ __forceinline__ int tiles_of(const Kv4Args& a, int L) {
  if (MODE == kDense) return (L + 15) >> 4;
  const Regions r = regions_of(L, a.ns, a.nl);
  if (MODE == kList) return (r.s_end + a.k + (L - r.l_start) + 15) >> 4;
  return r.l_start > r.s_end ? ((r.l_start + 15) >> 4) - (r.s_end >> 4) : 0;
}

__device__ __forceinline__ int len_of(const Kv4Args& a, int b) {
  const int L = a.seq_lens[b];
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

// The CTAs' shares.  A unit weighs its tiles and kUnit more, what entering and ending it takes of
// a CTA's time (short histories: a CTA of many units would be last by far); of the weight W, CTA
// c of n takes [W c / n, W (c + 1) / n), the tiles that lie there.  A unit's first kUnit places
// hold no tile.
constexpr int kUnit = 16, kLeast = 16;  // (a CTA weighs kLeast at least)
__device__ __forceinline__ long long quotient(long long x, long long y) {  // (64 bits: hundreds of cycles)
  return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
}
__device__ __forceinline__ long long share(long long W, int n, int c) { return quotient(W * c, n); }
__device__ __forceinline__ int holder(long long W, int n, long long place) { return (int)quotient((place + 1) * n - 1, W); }

struct Share {
  long long weight;  // of all units
  long long place;   // the first unit's, among the weights
  int ctas, tiles;   // CTAs that have a share; this one's tiles
};

// Every thread of the CTA gets the walk's length and the place where this CTA's share starts.  Either half
// of the threads sums the requests up, and the thread of each whose requests hold an end of the
// share finds the unit there (one after the other, the two ends take a microsecond).
template <int MODE, int W>
__device__ __forceinline__ Share find_share(const Kv4Args& a, Cursor* c) {
  constexpr int kHalf = 16 * W;
  __shared__ long long s_sum[2][W], s_tiles[2], s_place;
  __shared__ Cursor s_at;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, end = threadIdx.x >= kHalf ? 1 : 0;
  const int per = (a.B + kHalf - 1) / kHalf, b0 = (threadIdx.x - end * kHalf) * per, b1 = b0 + per < a.B ? b0 + per : a.B;
  long long tiles = 0, units = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = blockIdx.x == 0 && end == 0 ? load_len(a.seq_lens, b, a.max_len, a.status) : len_of(a, b);
    const int nt = tiles_of<MODE>(a, L);
    tiles += nt;
    units += nt > 0;
  }
  long long x = tiles, y = units;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long p = __shfl_up_sync(0xffffffffu, x, off), q = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) x += p, y += q;
  }
  if (lane == 31) s_sum[0][warp] = x, s_sum[1][warp] = y;
  if (threadIdx.x == 0) s_tiles[0] = s_tiles[1] = 0;
  __syncthreads();
  long long all = 0, all_units = 0;
  x -= tiles;
  y -= units;
  const int first = end * (W / 2), warps = a.B < kHalf ? (a.B + 31) >> 5 : W / 2;  // that have a request
#pragma unroll 1
  for (int w = first; w < first + warps; ++w) {
    if (w == warp) x += all, y += all_units;
    all += s_sum[0][w];
    all_units += s_sum[1][w];
  }
  Share r;
  r.weight = (all + kUnit * all_units) * a.H;
  long long n = (r.weight + kLeast - 1) / kLeast;  // (a power of two)
  n = n < 1 ? 1 : n > gridDim.x ? gridDim.x : n;
  r.ctas = (int)n;
  // the tiles before a share's ends: one thread's requests hold each
  const long long before = (x + kUnit * y) * a.H, after = before + (tiles + kUnit * units) * a.H;
  if (blockIdx.x < n) {
    const long long at = share(r.weight, (int)n, blockIdx.x + end);
    if (at == r.weight && threadIdx.x == kHalf) s_tiles[1] = all * a.H;
    if (at >= before && at < after) {
      long long off = at - before, t = x * a.H;
      for (int b = b0; b < b1; ++b) {
        const int L = len_of(a, b), nt = tiles_of<MODE>(a, L), w = nt > 0 ? nt + kUnit : 0;
        if (off < (long long)w * a.H) {
          const int h = (int)quotient(off, w), in = (int)(off - (long long)h * w), tile = in > kUnit ? in - kUnit : 0;
          s_tiles[end] = t + (long long)h * nt + tile;
          if (end == 0) {
            s_at.b = b;
            s_at.h = h;
            s_at.tile = tile;
            s_at.nt = nt;
            s_at.L = L;
            s_place = at - in;
          }
          break;
        }
        off -= (long long)w * a.H;
        t += (long long)nt * a.H;
      }
    }
  }
  __syncthreads();
  r.tiles = (int)(s_tiles[1] - s_tiles[0]);  // (a share has fewer tiles than 2^31)
  r.place = s_place;
  *c = s_at;
  return r;
}

// ---------------------------------------------------------------------------- a warp's ring
//
// Tile i of a CTA's share is warp i % W's.  A warp fetches its own tiles, S of them ahead, into a
// ring of its own: a stage is the cell of K, then the cell of V, as they lie in the pool.
// (A warp that feeds the others leaves them 96 registers of 128: the products spill.)

__device__ __forceinline__ void cp_async_cg16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Rows lie alone: of a line of 128 bytes, which L2 fetches otherwise, the half with the row (3,409 rows of
// 32K in lists, gathered: 91 -> 52 MB read of HBM).
template <int BYTES>
__device__ __forceinline__ void cp_async_row(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// (Plain loads here as of tables, lists and lengths: kernels start before those ahead of them on the stream end,
// and what these write is not constant for a kernel's whole life.)
template <int WORDS>
__device__ __forceinline__ void load_row(const void* src, uint32_t* w) {
  if constexpr (WORDS == 4)
    asm("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(src));
  else if constexpr (WORDS == 2)
    asm("ld.global.L2::64B.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(src));
  else
    asm("ld.global.L2::64B.u32 %0, [%1];" : "=r"(w[0]) : "l"(src));
}

// A lane's row on its way from its place in a list to its number.
struct Position {
  int t, lo, hi;   // as found, -1: none; where it has to lie
  uint32_t table;  // its row of the table
  int h;           // the pool's head
};
struct Entry {
  int e, off;  // its table entry; in the block, -1: none
  int h;
};

// of the j-th place of a unit's list
__device__ __forceinline__ void row_position(const Kv4Args& a, const Cursor& c, bool on, int j, Position& w) {
  w.t = -1;
  if (!on) return;
  const Regions g = regions_of(c.L, a.ns, a.nl);
  w.h = a.pool.hdiv == 1 ? c.h : c.h / a.pool.hdiv;
  w.table = a.pool.per_head ? (uint32_t)c.b * a.heads + w.h : c.b;
  w.lo = 0;
  w.hi = c.L;
  if (j < g.s_end) {
    w.t = j;
  } else if (j < g.s_end + a.k) {
    w.t = a.idx[((size_t)c.b * a.H + c.h) * a.k + (j - g.s_end)];
    w.lo = g.s_end;
    w.hi = g.l_start;
  } else {
    const int t = g.l_start + (j - g.s_end - a.k);
    w.t = t < c.L ? t : -1;
  }
}

__device__ __forceinline__ void row_entry(const Kv4Args& a, bool reports, const Position& p, Entry& w) {
  w.off = -1;
  if (p.t < 0) return;
  if (p.t < p.lo || p.t >= p.hi) {
    if (reports) flag(a.status, SKV_DEV_BAD_INDEX);
    return;
  }
  const int block = a.shift >= 0 ? p.t >> a.shift : p.t / a.bs;
  w.off = p.t - block * a.bs;
  w.h = p.h;
  w.e = a.pool.table[(size_t)p.table * a.pool.stride + block];
}

// The row's number in its pool, bit 31: the host's (pools have fewer than 2^31 rows).
constexpr uint32_t kNoRow = 0xffffffffu;
__device__ __forceinline__ uint32_t row_id(const Kv4Args& a, bool reports, const Entry& w) {
  if (w.off < 0) return kNoRow;
  if (w.e >= 0) {
    if ((uint32_t)w.e < a.n_gpu) return (a.pool.per_head ? w.e : w.e * a.heads + w.h) * a.bs + w.off;
  } else if (~(uint32_t)w.e < a.n_host) {
    return ((~(uint32_t)w.e * a.heads + w.h) * a.bs + w.off) | 0x80000000u;
  }
  if (reports) flag(a.status, SKV_DEV_BAD_SLOT);
  return kNoRow;
}

// Feeders.  issue() starts the next tile's copies, a commit group, into the ring's next stage; S - 1
// times at first, then once a tile before it is computed.  rows() then tells which of the 16 rows of the tile
// to be computed are there.  (Bulk copies with an mbarrier a stage cost more: the polls of a
// barrier take issue slots that the products need -- 8 requests of 32K keys, 95 us against 85.)

// A history's tiles: whole cells.  The warp finds 32 tiles at a time, a lane a tile; the entries of
// the next 32 are loaded when these are started.
template <int MODE, int NG, bool V, int W, int S>
struct CellFeeder {
  static constexpr int kCell = kv4_cell(NG), kStage = (V ? 2 : 1) * kCell;
  static constexpr uint32_t kNone = 0xffffffffu, kHost = 0x80000000u;
  const Kv4Args& a;
  Cursor& at;              // the next tile to be found (shared memory)
  uint32_t to, end;        // this lane's chunk of the next stage; past the last one
  uint32_t cell;           // this lane's tile: its cell's number in its pool
  int e;                   // its tile of the next 32: entry, the cell's number in block 0
  uint32_t in;
  int left, ahead, lane_up;  // tiles from these 32 on; not found; the lane whose tile is next
  uint32_t gone;             // of the tiles issued, the last in bit 0: no such block

  __device__ __forceinline__ CellFeeder(const Kv4Args& args, Cursor& at_, uint32_t*, uint32_t ring, Cursor c, int n)
      : a(args), at(at_), to(ring + (threadIdx.x & 31) * 16), end(to + S * kStage), cell(kNone), e(0), in(kNone), left(n), ahead(n), lane_up(0),
        gone(0) {
    if ((threadIdx.x & 31) == 0) at = c;
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) turn();
  }
  // the next 32 tiles' places and entries
  __device__ __forceinline__ void find() {
    const int lane = threadIdx.x & 31;
    Cursor c = at;
    __syncwarp();
    c.tile += lane * W;
    in = kNone;
    if (lane < ahead) {
      settle<MODE>(a, c);
      const int i = (MODE == kScore ? regions_of(c.L, a.ns, a.nl).s_end >> 4 : 0) + c.tile;
      const int block = a.shift >= 0 ? i >> (a.shift - 4) : i / a.cells;
      in = c.h * a.cells + (i - block * a.cells);
      e = table_row(a.pool, c.b, c.h, a.heads)[block];
      if (a.pool.per_head && e >= 0) in -= c.h * a.cells;
      if (lane == 31) {
        c.tile += W;
        at = c;
      }
    }
    __syncwarp();
    ahead -= 32;
  }
  // what was found becomes what is issued
  __device__ __forceinline__ void turn() {
    cell = kNone;
    if (in != kNone) {
      if ((unsigned)e < a.n_gpu)
        cell = (unsigned)e * a.block_cells + in;
      else if (e < 0 && ~(unsigned)e < a.n_host)
        cell = (~(unsigned)e * (unsigned)(a.heads * a.cells) + in) | kHost;
      else
        flag(a.status, SKV_DEV_BAD_SLOT);
    }
    find();
  }
  __device__ __forceinline__ void copy(const void* kp, const void* vp, uint32_t c) {
    const int lane = threadIdx.x & 31;
    const size_t off = (size_t)c * kCell + lane * 16;
    const unsigned char *k = (const unsigned char*)kp + off, *v = (const unsigned char*)vp + off;
    cp_async_cg16(to, k);
    cp_async_cg16(to + 512, k + 512);
    if (V) {
      cp_async_cg16(to + kCell, v);
      cp_async_cg16(to + kCell + 512, v + 512);
    }
    if (lane < 4 * NG) {
      cp_async_cg16(to + 1024, k + 1024);
      if (V) cp_async_cg16(to + kCell + 1024, v + 1024);
    }
  }
  __device__ __forceinline__ void issue() {
    gone <<= 1;
    if (lane_up < left) {
      if (lane_up == 32) {
        left -= 32;
        lane_up = 0;
        turn();
      }
      const uint32_t c = __shfl_sync(0xffffffffu, cell, lane_up++);
      if (c < kHost)
        copy(a.pool.gpu_k, a.pool.gpu_v, c);
      else if (c != kNone)
        copy(a.pool.host_k, a.pool.host_v, c & ~kHost);
      else
        gone |= 1u;
    }
    cp_async_commit();
    to = to + kStage == end ? end - S * kStage : to + kStage;
  }
  // of the tile S - 1 issues ago, n rows before its request's end
  __device__ __forceinline__ uint32_t rows(int n, int) const {
    return gone >> (S - 1) & 1u ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1u;
  }
};

// A list's tiles: rows, by 16-byte copies.  A lane finds a row of two tiles (this warp's next and the one
// after) in three steps -- its place's position, that one's entry, the row -- so each load has two
// tiles' time to arrive.
template <int NG, int W, int S>
struct RowFeeder {
  static constexpr int kCell = kv4_cell(NG), kStage = 2 * kCell;
  const Kv4Args& a;
  uint32_t* masks;
  uint32_t to, end;  // the next stage; past the last one
  Cursor c;  // this half warp's next tile
  int left, half;
  uint32_t row;  // this lane's, of the tiles that are issued; then: position on its way, entry on its way
  Position position;
  Entry entry;

  __device__ __forceinline__ RowFeeder(const Kv4Args& args, Cursor&, uint32_t* masks_, uint32_t ring_, Cursor at, int n)
      : a(args), masks(masks_), to(ring_), end(ring_ + S * kStage), c(at), left(n), half(-2), row(kNoRow) {
    c.tile += (threadIdx.x >> 4 & 1) * W;
    left -= threadIdx.x >> 4 & 1;
    position.t = entry.off = -1;
  }
  __device__ __forceinline__ void issue() {
    const int lane = threadIdx.x & 31;
    if (half <= 0) {  // (at the start: three times)
#pragma unroll 1
      for (; half <= 0; ++half) {
        row = row_id(a, true, entry);
        row_entry(a, true, position, entry);
        if (left > 0 && c.tile >= c.nt) settle<kList>(a, c);
        row_position(a, c, left > 0, (c.tile << 4) + (lane & 15), position);
        left -= 2;
        c.tile += 2 * W;
      }
      half = 0;
    }
    const uint32_t live = __ballot_sync(0xffffffffu, row != kNoRow) >> (16 * half) & 0xffffu;
    if (lane == 0) masks[(to - (end - S * kStage)) / kStage] = live;
    auto at = [&](uint32_t r, bool v) {  // the row's cell
      const unsigned char* base = (const unsigned char*)(r >> 31 ? (v ? a.pool.host_v : a.pool.host_k)
                                                                 : (v ? a.pool.gpu_v : a.pool.gpu_k));
      return base + (size_t)(r >> 4 & 0x7ffffffu) * kCell;
    };
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // rows 8 j .. 8 j + 7, four lanes each
      const uint32_t r = __shfl_sync(0xffffffffu, row, (lane >> 2) + 8 * j + 16 * half);
      if (r != kNoRow) {
        const int off = (int)(r & 15u) * kCodeBytes + (lane & 3) * 16;
        cp_async_row<16>(to + lane * 16 + 512 * j, at(r, false) + off);
        cp_async_row<16>(to + kCell + lane * 16 + 512 * j, at(r, true) + off);
      }
    }
    const uint32_t r = __shfl_sync(0xffffffffu, row, (lane & 15) + 16 * half);
    if (r != kNoRow) {  // K's words, V's
      const uint32_t dst = to + (lane >> 4) * kCell + 16 * kCodeBytes + (lane & 15) * 4 * NG;
      const unsigned char* src = at(r, lane >= 16) + 16 * kCodeBytes + (r & 15u) * 4 * NG;
      cp_async_row<4 * NG>(dst, src);
    }
    cp_async_commit();
    half = half == 0 ? 1 : 0;
    to = to + kStage == end ? end - S * kStage : to + kStage;
  }
  __device__ __forceinline__ uint32_t rows(int, int stage) const { return masks[stage]; }
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// the larger magnitudes of two pairs (a NaN gives way)
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.f16x2 %0, x, y;\n\t}" : "=r"(r) : "r"(a), "r"(b));
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
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 u = lds128(addr);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = lds64(addr);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = lds32(addr);
  }
}
__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float centre_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The four operand registers of two bytes' worth of codes, in the order low and high half of
// the first byte, low and high half of the second: subnormal fp16 pairs, 2^-24 and 2^-20 a unit.  The second byte,
// brought down by a permutation that clears what is above it, is a subnormal itself, and BYTE leaves it in the
// high half's place: 16 high + low, 2^-24 a unit, of which a sum of products gives the low
// half's back once at the end (a mask a register less: a million keys 211 -> 204 us).
template <bool BYTE>
__device__ __forceinline__ void spread(uint32_t x, uint32_t* r) {
  const uint32_t y = __byte_perm(x, 0u, 0x4341);
  r[0] = x & 0x000f000fu;
  r[1] = x & 0x00f000f0u;
  r[2] = y & 0x000f000fu;
  r[3] = BYTE ? y : y & 0x00f000f0u;
}

// A power of two that brings |x| <= mx under 2^10 (its own inverse is exact too).
__device__ __forceinline__ float fit(float mx) {
  int e = 263 - (int)((__float_as_uint(mx) >> 23) & 255u);
  e = e < 1 ? 1 : e > 254 ? 254 : e;
  return __uint_as_float((uint32_t)e << 23);
}

// Queries as the second operand: columns are heads, k-steps 16 entries in the order that the codes
// come in; wz: the group sums, three bf16 parts, against words.  Groups of 32: k-step j has
// the entries 16 j .. 16 j + 15, a lane's register of codes one byte each of its two runs of eight.
// Larger groups: k-step 4 a + 2 b + c has of the spans 4 a + c and 4 a + c + 2 the
// bytes b of each lane, and a register of codes comes from one word as it is (a million keys in groups
// of 128: 215 -> 211 us).
template <int NT>
struct QFrag {
  uint32_t b[NT][8][2];
  uint32_t wz[NT][3];
  float unit[NT][2];  // what a logit of heads 2 t, 2 t + 1 comes in: 2^20 / their power of two
};

// A CTA makes them together, warp j < 8 the j-th k-step, and every warp takes its lanes' copies.
template <int NT>
struct QShared {
  uint32_t b[NT][8][2][32], wz[NT][3][32];
  float largest[8 * NT][8], part[8][8 * NT];  // of a head: of each warp's entries; sums of a k-step
};

// This warp's k-step of the columns: entries 16 warp + 4 t .. of head 8 nt + g.  MEAN: of the heads' sum.
template <int NT, bool MEAN>
__device__ __forceinline__ void load_queries(const __nv_bfloat16* q, int n, float (&x)[NT][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[nt][i] = 0.f;
    const int head = 8 * nt + g;
    constexpr int kTogether = MEAN ? 4 : 1;  // loads on their way
#pragma unroll 1
    for (int h = MEAN ? 0 : head; h < n && warp < 8; h += kTogether) {
      uint2 u[kTogether];
#pragma unroll
      for (int k = 0; k < kTogether; ++k)
        u[k] = h + k < n ? *reinterpret_cast<const uint2*>(q + (size_t)(h + k) * kD + 16 * warp + 4 * t) : make_uint2(0u, 0u);
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        x[nt][0] += __uint_as_float(u[k].x << 16);
        x[nt][1] += __uint_as_float(u[k].x & 0xffff0000u);
        x[nt][2] += __uint_as_float(u[k].y << 16);
        x[nt][3] += __uint_as_float(u[k].y & 0xffff0000u);
      }
      if (!MEAN) break;
    }
  }
}

// MEAN: the mean of the n heads in three fp16 parts, columns 0, 1 and 2; else a column a head.
template <int NG, int NT, bool MEAN>
__device__ __forceinline__ void make_queries(float (&x)[NT][4], int n, QShared<NT>& s, QFrag<NT>& f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = 8 * nt + g;
    if (MEAN) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] /= (float)n;
    }
    float m = fmaxf(fmaxf(fabsf(x[nt][0]), fabsf(x[nt][1])), fmaxf(fabsf(x[nt][2]), fabsf(x[nt][3])));
    float sum = (x[nt][0] + x[nt][1]) + (x[nt][2] + x[nt][3]);
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
    }
    if (t == 0 && warp < 8) {
      s.largest[head][warp] = m;
      s.part[warp][head] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = 8 * nt + g;
    const float4* lg = reinterpret_cast<const float4*>(s.largest[head]);
    const float4 u = lg[0], v = lg[1];
    const float scale = fit(fmaxf(fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)), fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w))));
    const float unit = 0x1p20f / scale;
    f.unit[nt][0] = __shfl_sync(0xffffffffu, unit, 8 * t);
    f.unit[nt][1] = __shfl_sync(0xffffffffu, unit, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y = x[nt][i] * scale;
      if (MEAN) {
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
          const float h = __half2float(__float2half_rn(y));
          if (k == g) x[nt][i] = h;
          y -= h;
        }
        if (g >= 3) x[nt][i] = 0.f;
      } else {
        x[nt][i] = y;
      }
    }
    if (warp < 8) {
      if (NG == 4) {
        s.b[nt][warp][0][lane] = pack_f16(16.f * x[nt][0], 16.f * x[nt][2]);
        s.b[nt][warp][1][lane] = pack_f16(x[nt][1], x[nt][3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<__half*>(&s.b[nt][(warp & 4) + (i & 2) + (warp & 1)][i & 1][lane])[warp >> 1 & 1] =
              __float2half_rn(i & 1 ? x[nt][i] : 16.f * x[nt][i]);
      }
    }
    if (warp == 0) {  // the t-th group's sum, in the products' unit
      float z = 0.f;
      if (t < NG && (!MEAN || g == 0)) {
#pragma unroll 1
        for (int j = t * 8 / NG; j < (t + 1) * 8 / NG; ++j) z += s.part[j][head];
      }
      z *= scale * 0x1p-20f;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const float h = __bfloat162float(__float2bfloat16_rn(z));
        s.wz[nt][i][lane] = tc::pack_bf16(-8.f * h, h);
        z -= h;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.b[nt][j][0] = s.b[nt][j][0][lane], f.b[nt][j][1] = s.b[nt][j][1][lane];
#pragma unroll
    for (int i = 0; i < 3; ++i) f.wz[nt][i] = s.wz[nt][i][lane];
  }
}

// The key of the operands' row r: every second pair exchanged, so that the 16-byte loads of K's
// codes meet no bank twice (rows 2 i and 2 i + 1 half a line apart) and the 8-byte loads of V's,
// at rows 0, 2, 4, 6, only in pairs.
__device__ __forceinline__ int key_of(int r) { return r ^ (r >> 1 & 1); }

// The logits of a cell, in the columns' units: c[nt][0..1] key key_of(g) of heads 2 t, 2 t + 1; [2..3]
// the key 8 on.  A row's logits depend on that row alone: those of rows that are not there are anything.
template <int NG, int NT>
__device__ __forceinline__ void logits(uint32_t cell, const QFrag<NT>& f, float (&c)[NT][4]) {
  const int lane = threadIdx.x & 31, g = key_of(lane >> 2), t = lane & 3;
  const uint4 k0 = lds128(cell + g * kCodeBytes + t * 16), k1 = lds128(cell + (g + 8) * kCodeBytes + t * 16);
  const uint32_t words = cell + 16 * kCodeBytes;
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
  for (int jj = 0; jj < 4; ++jj) {  // two k-steps
    uint32_t r0[4], r1[4];
    auto codes = [&](const uint4& k) {
      const uint32_t x = jj < 2 ? k.x : k.y, z = jj < 2 ? k.z : k.w;
      return NG == 4 ? __byte_perm(x, z, jj & 1 ? 0x7632u : 0x5410u) : jj & 1 ? z : x;
    };
    spread<false>(codes(k0), r0);
    spread<false>(codes(k1), r1);
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

// A warp's state of a unit: p_t = 2^(x_t + ref), ref = -27 - the running maximum, whole numbers.  (A weight is
// 2^-20 at the most and their sum under 2^10 whatever the keys: values up to 2^116 times it stay in fp32.)  The operand of a
// key, head and group, w = p s 2^e, has a power of two of its own, which keeps the largest one so far
// between 2^7 and 2^15: fp16 holds it to 11 bits, and what lies under 2^-21 of that largest to 2^-32 of it.  (A power
// that heads or groups share goes by the largest product of all, and others' may be lost.)
template <int NG, int NT>
struct State {
  float l[NT][2], ref[NT][2];
  float top[NT][2];   // the logit, in its column's unit, past which the maximum moves
  // rows 2 g (2^-24 a unit) and 2 g + 1 (2^-20; i odd: 16 of it and the other, 2^-24) of entries
  // 16 i, columns heads 2 t, 2 t + 1; times 2^e
  float o[NT][8][4];
  float z[NT][NG][2];
  float pw[NT][NG][2];  // 2^e; negative where this lane's keys are the complemented ones
};
constexpr float kFloor = -3.0e38f;
// e ends here: weights times it stay in fp32, and steps from 2^-75 up have their largest operand at 2^7.  (It begins
// at -97: a product lies below 2^105.)
constexpr int kPowMax = 110;
constexpr int kShift = 27;

__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }
__device__ __forceinline__ float power_of(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(e + 127) << 23); }

// of a sum of weights l under the reference -m
__device__ __forceinline__ float lse_of(float m, float l) { return kLn2 * ((m - (float)kShift) + log2f(l * power_of(kShift))); }

template <int NG, int NT>
__device__ __forceinline__ void clear(State<NG, NT>& s) {
  const float pw = threadIdx.x & 4 ? -power_of(kPowMax) : power_of(kPowMax);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.l[nt][i] = 0.f;
      s.ref[nt][i] = -kFloor;
      s.top[nt][i] = kFloor;
#pragma unroll
      for (int g = 0; g < NG; ++g) s.z[nt][g][i] = 0.f, s.pw[nt][g][i] = pw;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s.o[nt][i][j] = 0.f;
  }
}

// A logit of the cell has passed its head's maximum by 2^7: that head's sums in a new reference.  All factors are powers
// of two.  The operands' powers take up the difference, so that the outputs stay -- but for what
// would take them past their end.
template <int NG, int NT>
__device__ __forceinline__ void move_maximum(State<NG, NT>& s, const float (&c)[NT][4], const float (&kf)[NT][2]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float m = fmaxf(c[nt][i], c[nt][i + 2]);
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (m > s.top[nt][i]) {
        m = ceilf(m * kf[nt][i]);
        const float ref = -(float)kShift - m, down = fmaxf(ref - s.ref[nt][i], -1000.f), f = power_of((int)down);
        const bool first = s.ref[nt][i] == -kFloor;
        s.ref[nt][i] = ref;
        s.top[nt][i] = (m + 7.f) / kf[nt][i];
        if (first) continue;  // (nothing to bring down)
        s.l[nt][i] *= f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          s.z[nt][g][i] *= f;
          const int room = kPowMax - exponent_of(s.pw[nt][g][i]), up = min((int)-down, room);
          s.pw[nt][g][i] = __uint_as_float(__float_as_uint(s.pw[nt][g][i]) + ((uint32_t)up << 23));
          if (up < (int)-down) {
            const float k = power_of((int)down + up);
#pragma unroll
            for (int j = g * 8 / NG; j < (g + 1) * 8 / NG; ++j) s.o[nt][j][i] *= k, s.o[nt][j][i + 2] *= k;
          }
        }
      }
    }
}

// An operand of the cell has reached 2^15: its head's and group's power of two goes down, and the outputs with it.
template <int NG, int NT>
__device__ __forceinline__ void lower_powers(State<NG, NT>& s, const float (&p)[NT][4], const uint32_t (&w0)[NG], const uint32_t (&w1)[NG]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float m = fmaxf(p[nt][i] * fabsf(step_of(w0[g])), p[nt][i + 2] * fabsf(step_of(w1[g])));
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (m * fabsf(s.pw[nt][g][i]) >= 0x1p15f) {
          const int e = 7 - exponent_of(m);
          const float k = power_of(e - exponent_of(s.pw[nt][g][i]));
          s.pw[nt][g][i] = copysignf(power_of(e), s.pw[nt][g][i]);
#pragma unroll
          for (int j = g * 8 / NG; j < (g + 1) * 8 / NG; ++j) s.o[nt][j][i] *= k, s.o[nt][j][i + 2] *= k;
        }
      }
}

// The cell's operands, keys by heads; true where one has reached 2^15.
template <int NG, int NT>
__device__ __forceinline__ bool weigh(const State<NG, NT>& s, const float (&p)[NT][4], const uint32_t (&w0)[NG], const uint32_t (&w1)[NG],
                                      uint32_t (&w)[NT][NG][2]) {
  uint32_t most = 0u;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float s0 = step_of(w0[g]), s1 = step_of(w1[g]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {  // (the power first: a weight that is 0 stays 0 whatever the step)
      const float2 e = make_float2(s.pw[nt][g][0], s.pw[nt][g][1]);
      const float2 x = mul2(mul2(make_float2(p[nt][0], p[nt][1]), e), make_float2(s0, s0));
      const float2 y = mul2(mul2(make_float2(p[nt][2], p[nt][3]), e), make_float2(s1, s1));
      w[nt][g][0] = pack_f16(x.x, x.y);
      w[nt][g][1] = pack_f16(y.x, y.y);
      most = max_abs(most, max_abs(w[nt][g][0], w[nt][g][1]));
    }
  }
  return (most + 0x08000800u) & 0x80008000u;
}

// A cell's keys into the state.  The weights p_t meet the centres in fp32 and, times the steps, the
// codes on the tensor core.  Every other row's codes come as 15 - c and its weights negative:
// w c - w' (15 - c') + 15 w'.  Codes are 7.5 on average, and a long sum of them on one side of zero would lose
// to the tensor core's truncation what the centring takes off again (a million keys: 1 % of the
// output).  With the codes' own 8, the even keys' stand 8 too high and the odd ones' 7 too low.
template <int NG, int NT>
__device__ __forceinline__ void attend_cell(uint32_t cell, uint32_t mask, const QFrag<NT>& f, const float (&kf)[NT][2],
                                            State<NG, NT>& s) {
  constexpr int kCell = kv4_cell(NG);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, key = key_of(g);
  float c[NT][4];
  logits<NG, NT>(cell, f, c);
  const uint32_t words = cell + kCell + 16 * kCodeBytes;
  uint32_t w0[NG], w1[NG];
  lds_words<NG>(words + key * 4 * NG, w0);
  lds_words<NG>(words + (key + 8) * 4 * NG, w1);
  if (mask != 0xffffu) {  // what lies in rows that are not there counts for nothing
    const bool on0 = mask >> key & 1u, on1 = mask >> (key + 8) & 1u;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      w0[i] = on0 ? w0[i] : 0u;
      w1[i] = on1 ? w1[i] : 0u;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[nt][i] = (i < 2 ? on0 : on1) ? c[nt][i] : -INFINITY;
  }
  bool past = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) past |= fmaxf(c[nt][i], c[nt][i + 2]) > s.top[nt][i];
  if (__any_sync(0xffffffffu, past)) move_maximum<NG, NT>(s, c, kf);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[nt][i] = ex2(fmaf(c[nt][i], kf[nt][i & 1], s.ref[nt][i & 1]));
    s.l[nt][0] += c[nt][0] + c[nt][2];
    s.l[nt][1] += c[nt][1] + c[nt][3];
  }
  // (what does not wait for the operands' vote comes before it: a million keys 204.9 us behind it, 202.2 so)
  uint32_t w[NT][NG][2];
  const bool past_range = weigh<NG, NT>(s, c, w0, w1, w);
  const float off = g & 1 ? 7.f : -8.f;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const float y0 = fmaf(off, step_of(w0[i]), centre_of(w0[i])), y1 = fmaf(off, step_of(w1[i]), centre_of(w1[i]));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      s.z[nt][i][0] = fmaf(c[nt][0], y0, fmaf(c[nt][2], y1, s.z[nt][i][0]));
      s.z[nt][i][1] = fmaf(c[nt][1], y0, fmaf(c[nt][3], y1, s.z[nt][i][1]));
    }
  }
  uint2 v[4];
  {  // the keys of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9: two apart from each other's, in one order or the other
    const uint32_t row = cell + kCell + 2 * t * kCodeBytes + (g << 3), even = (t & 1) * kCodeBytes, odd = kCodeBytes - even;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds64(row + (i & 1 ? odd : even) + (i >> 1) * 8 * kCodeBytes);
    v[1] = make_uint2(~v[1].x, ~v[1].y);
    v[3] = make_uint2(~v[3].x, ~v[3].y);
  }
  if (__any_sync(0xffffffffu, past_range)) {
    lower_powers<NG, NT>(s, c, w0, w1);
    weigh<NG, NT>(s, c, w0, w1, w);
  }
  uint32_t wb[NT][2];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    const uint32_t sel = jj & 1 ? 0x7632u : 0x5410u;
    uint32_t r0[4], r1[4];
    spread<true>(__byte_perm(jj < 2 ? v[0].x : v[0].y, jj < 2 ? v[1].x : v[1].y, sel), r0);
    spread<true>(__byte_perm(jj < 2 ? v[2].x : v[2].y, jj < 2 ? v[3].x : v[3].y, sel), r1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 2 * jj + i;
      constexpr int kSteps = 8 / NG;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (j % kSteps == 0) {
          wb[nt][0] = tc::movmatrix_t(w[nt][j / kSteps][0]);
          wb[nt][1] = tc::movmatrix_t(w[nt][j / kSteps][1]);
        }
        const uint32_t ar[4] = {r0[2 * i], r0[2 * i + 1], r1[2 * i], r1[2 * i + 1]};
        mma_f16(s.o[nt][j], ar, wb[nt][0], wb[nt][1]);
      }
    }
  }
}

template <int NG, int NT, int MODE>
struct AttnShape {
  // Warps of a CTA, CTAs a SM, stages of 2.2 to 2.5 KB a warp.  One CTA a SM: of two, the schedulers serve
  // the one that came first before the other, it ends at 80 % of the time and leaves the SM half empty
  // (a million keys in groups of 128, 8 warps in either: 231 us; 12 or 16 warps in one 215, 8 warps
  // 258).  16 warps have 128 registers each, 12 have 168: groups of 128 fit in the first (211 us with
  // 12, 201 with 16), those of 32 and 64 do not (8 requests of 32K: 78 us with 12, 82 with 16).  A
  // list's rows arrive late rather, and two CTAs hide more of that (3,409 rows of 32K for 8 requests:
  // 26.8 us, one CTA 28.8), although groups of 32 and 64 spill there (100 and 12 bytes a thread).  Two column
  // tiles take all the registers of 8 warps.
  static constexpr int kCtas = NT == 1 && MODE == kList ? 2 : 1;
  static constexpr int kW = NT == 2 || MODE == kList ? 8 : NG == 1 ? 16 : 12;
  static constexpr int kStages = NT == 2 ? 6 : MODE == kList || NG == 1 ? 3 : 5;
  static constexpr int kRing = kW * kStages * 2 * kv4_cell(NG);
  static constexpr int kRow = kD + 4;  // floats of a head's partial row: heads 2 t, 2 t + 2 an eighth of the banks apart
  static constexpr int kOut = kW * 8 * NT * kRow * 4;
  static constexpr int kSmem = kRing + kOut;
};

template <int MODE, int NG, int W, int S>
struct Pick {
  using type = CellFeeder<MODE, NG, true, W, S>;
};
template <int NG, int W, int S>
struct Pick<kList, NG, W, S> {
  using type = RowFeeder<NG, W, S>;
};

// Persistent CTAs, a share each of the tiles of all units; a warp computes its own tiles.  Measured
// (8 KV heads): 8 requests of 32K keys in groups of 32, 8 query heads each, 336 MB, 75 us (4.5 TB/s); a
// million keys in groups of 128, 4 query heads, 1,141 MB, 199 us (5.7 TB/s); lists of 3,409 rows of 32K
// for the 8 requests, 52 MB read, 24.5 us; 4 requests to 777 keys 11.3 us a call.  The instructions of
// a tile and how they wait for each other bound it: 360 in groups of 32, 154 of them masks, permutations and
// shifts at half the issue rate, and 18 products, at 60 % of the issue slots; the copies alone take 60
// (a million keys: 178).  4 us pass before the first product: lengths, the share's ends, table, cells.
template <int NG, int NT, int MODE>
__global__ void __launch_bounds__(32 * AttnShape<NG, NT, MODE>::kW, AttnShape<NG, NT, MODE>::kCtas) kv4_attn_kernel(const Kv4Args a) {
  using Shape = AttnShape<NG, NT, MODE>;
  constexpr int W = Shape::kW, S = Shape::kStages, HC = 8 * NT;  // columns
  constexpr int kStage = 2 * kv4_cell(NG);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Cursor s_at[W];
  __shared__ uint32_t s_mask[MODE == kList ? W : 1][S];
  __shared__ float2 s_ml[HC][W];
  __shared__ __align__(16) QShared<NT> s_q;
  // the walk's state between units, which the products need no registers for
  __shared__ Cursor s_unit;
  __shared__ long long s_at_place;  // of the unit among the weights
  float* s_o = reinterpret_cast<float*>(smem + Shape::kRing);
  pdl_release();
  pdl_wait();
  Cursor at;
  const Share mine = find_share<MODE, W>(a, &at);
  if (mine.tiles == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int share = mine.tiles;
  const uint32_t ring = smem_u32(smem) + warp * S * kStage;
  auto queries = [&](const Cursor& u) { return a.q + ((size_t)u.b * a.Hq + (size_t)u.h * a.G) * kD; };
  float x[NT][4];
  load_queries<NT, false>(queries(at), a.G, x);
  if (threadIdx.x == 0) {
    s_unit = at;
    s_at_place = mine.place;
  }
  at.tile += warp;
  typename Pick<MODE, NG, W, S>::type feed(a, s_at[warp], s_mask[MODE == kList ? warp : 0], ring, at,
                                        share > warp ? (share - warp + W - 1) / W : 0);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) feed.issue();
  int stage = 0, next = warp;  // this warp's next tile
  __syncthreads();
  // units of the share: tiles [from, to) of it, the unit's first at `base`
  for (int from = 0, seg = 0; from < share; ++seg) {
    const int base = from - s_unit.tile, left = s_unit.nt - s_unit.tile, to = left < share - from ? from + left : share;
    const uint32_t rows = (uint32_t)s_unit.L + 16u * (uint32_t)base;  // where the unit's rows end, 16 a tile from the share's first
    QFrag<NT> q;
    float kf[NT][2];
    State<NG, NT> s;
    clear(s);
    if (seg > 0) load_queries<NT, false>(queries(s_unit), a.G, x);
    make_queries<NG, NT, false>(x, a.G, s_q, q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) kf[nt][i] = fmaxf(q.unit[nt][i] * a.scale_log2, 0x1p-126f);  // (0 times -inf: NaN)
    // this warp's tiles
#pragma unroll 1
    for (; next < to; next += W) {
      cp_async_wait<S - 2>();
      __syncwarp();
      feed.issue();  // into the stage of the tile before this one
      const uint32_t mask = feed.rows((int)(rows - 16u * (uint32_t)next), stage);
      if (mask != 0u) attend_cell<NG, NT>(ring + stage * kStage, mask, q, kf, s);
      stage = stage == S - 1 ? 0 : stage + 1;
    }
    // the warp's sums and its output under its own reference; the CTA's below
#pragma unroll 1
    for (int off = 4; off <= 16; off <<= 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s.l[nt][i] += __shfl_xor_sync(0xffffffffu, s.l[nt][i], off);
#pragma unroll
          for (int k = 0; k < NG; ++k) s.z[nt][k][i] += __shfl_xor_sync(0xffffffffu, s.z[nt][k][i], off);
        }
    }
    float* row = s_o + warp * HC * Shape::kRow + 2 * g;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = 8 * nt + 2 * t + i;
        if (g == 0) s_ml[head][warp] = make_float2(-s.ref[nt][i], s.l[nt][i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = s.z[nt][j * NG / 8][i], lo = s.o[nt][j][i], hi = s.o[nt][j][i + 2];
          const float unit = power_of(24 - exponent_of(s.pw[nt][j * NG / 8][i]));
          *reinterpret_cast<float2*>(row + head * Shape::kRow + 16 * j) =
              make_float2(fmaf(lo, unit, z), fmaf(j & 1 ? hi - lo : hi, 0x1p-4f * unit, z));
        }
      }
    __syncthreads();
    const Cursor u = s_unit;
    const bool whole = base >= 0 && base + u.nt <= share;
    const size_t hq = (size_t)u.b * a.Hq + (size_t)u.h * a.G;
    float* slot = a.ws + ((size_t)blockIdx.x * 2 + (seg > 0)) * kSlotFloats;
    const int d = threadIdx.x & (kD - 1);
#pragma unroll 1
    for (int head = threadIdx.x / kD; head < a.G; head += 32 * W / kD) {
      float2 x[W];
      float m = kFloor, l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x[w] = s_ml[head][w];
        m = fmaxf(m, x[w].x);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float fw = ex2(x[w].x - m);
        l = fmaf(fw, x[w].y, l);
        o = fmaf(fw, s_o[(w * HC + head) * Shape::kRow + d], o);
      }
      if (whole) {
        a.out[(hq + head) * kD + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
        if (d == 0 && a.lse) a.lse[hq + head] = l == 0.f ? -INFINITY : lse_of(m, l);
      } else {
        slot[head * kD + d] = o;
        if (d == 0) *reinterpret_cast<float2*>(slot + 16 * kD + 2 * head) = make_float2(m, l);
      }
    }
    if (threadIdx.x == 0 && base >= 0)
      a.desc[(size_t)u.b * a.H + u.h] =
          make_int2((int)blockIdx.x | (seg > 0 ? 1 << 30 : 0), holder(mine.weight, mine.ctas, s_at_place + kUnit + u.nt - 1));
    __syncthreads();
    from = to;
    if (from < share) {
      if (threadIdx.x == 0) {
        s_at_place += kUnit + u.nt;
        Cursor n = u;
        n.tile = n.nt;
        settle<MODE>(a, n);
        s_unit = n;
      }
      __syncthreads();
    }
  }
}

// The units that no CTA held alone: their partials joined, a CTA a head; the empty ones: zeros; the others' CTAs
// return (of many short requests that is most of the grid).  A launch and two
// loads' latency, 2 us behind the attention's last CTA (by the last CTA to finish, it would need counters that
// somebody zeroes).
template <int MODE>
__global__ void __launch_bounds__(kD) kv4_merge_kernel(const Kv4Args a) {
  __shared__ float2 s_ml[kMaxParts];
  __shared__ float s_red[kD / 32];
  pdl_release();
  pdl_wait();
  const long long unit = blockIdx.x / a.G;
  const int head = blockIdx.x - (int)unit * a.G, b = (int)(unit / a.H), h = (int)(unit - (long long)b * a.H);
  const int d = threadIdx.x, lane = d & 31, warp = d >> 5;
  const size_t hq = (size_t)b * a.Hq + (size_t)h * a.G + head;
  const int2 span = a.desc[unit];  // (of an empty unit: anything)
  if (tiles_of<MODE>(a, len_of(a, b)) == 0) {
    a.out[hq * kD + d] = __float2bfloat16_rn(0.f);
    if (d == 0 && a.lse) a.lse[hq] = -INFINITY;
    return;
  }
  const int c0 = span.x & ((1 << 30) - 1), parts = span.y - c0 + 1;
  if (parts == 1) return;
  const float* slots = a.ws + (size_t)c0 * 2 * kSlotFloats + head * kD + d;
  const float2* sums = reinterpret_cast<const float2*>(a.ws + (size_t)c0 * 2 * kSlotFloats + 16 * kD + 2 * head);
  const size_t first = span.x >> 30 ? kSlotFloats : 0;  // the others begin with this unit
  auto at = [&](int i) { return i == 0 ? first : (size_t)i * 2 * kSlotFloats; };
  constexpr int kAhead = 8;  // outputs on their way beside the sums
  float ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ahead[i] = i < parts ? __ldcg(slots + at(i)) : 0.f;
  float m = kFloor;
  for (int i = d; i < parts; i += kD) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(reinterpret_cast<const float*>(sums) + at(i)));
    s_ml[i] = v;
    m = fmaxf(m, v.x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) s_red[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kD / 32; ++w) m = fmaxf(m, s_red[w]);
  float l = 0.f, o = 0.f;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < parts) {
      const float2 v = s_ml[i];
      const float f = ex2(v.x - m);
      l = fmaf(f, v.y, l);
      o = fmaf(f, ahead[i], o);
    }
#pragma unroll 8
  for (int i = kAhead; i < parts; ++i) {
    const float2 v = s_ml[i];
    const float f = ex2(v.x - m);
    l = fmaf(f, v.y, l);
    o = fmaf(f, __ldcg(slots + at(i)), o);
  }
  a.out[hq * kD + d] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  if (d == 0 && a.lse) a.lse[hq] = l == 0.f ? -INFINITY : lse_of(m, l);
}

// ---------------------------------------------------------------------------- scores

// Warps of a CTA, CTAs a SM, stages of 1.25 KB a warp.  (8 requests of 32K: 41 us; three CTAs: 45.)
constexpr int kScoreW = 8, kScoreCtas = 2, kScoreStages = 6;

// 8 requests of 32K keys in groups of 32, 8 KV heads of 8: 167 MB read, 39 us a call, 4.5 TB/s.  Of 41 in a
// graph, 36 without the products, 34 without the stores too, 39.5 on cells from L2: a start of 5 us, then HBM and the
// 194 instructions of a tile at 60 % of the issue slots, neither hidden by the other entirely.
template <int NG, int NT, int AGG>
__global__ void __launch_bounds__(32 * kScoreW, kScoreCtas) kv4_score_kernel(const Kv4Args a) {
  constexpr int W = kScoreW, S = kScoreStages, kCell = kv4_cell(NG);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Cursor s_at[W];
  __shared__ __align__(16) QShared<NT> s_q;
  pdl_release();
  pdl_wait();
  Cursor u;
  const Share mine = find_share<kScore, W>(a, &u);
  if (mine.tiles == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = key_of(lane >> 2), t = lane & 3;
  const int share = mine.tiles;
  Cursor at = u;
  at.tile += warp;
  const uint32_t ring = smem_u32(smem) + warp * S * kCell;
  auto queries = [&]() { return a.q + ((size_t)u.b * a.H + u.h) * a.Gi * kD; };
  float x[NT][4];
  load_queries<NT, AGG == SKV_AGG_MEAN>(queries(), a.Gi, x);
  CellFeeder<kScore, NG, false, W, S> feed(a, s_at[warp], nullptr, ring, at, share > warp ? (share - warp + W - 1) / W : 0);
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) feed.issue();
  int stage = 0, next = warp;
  for (int from = 0; from < share;) {
    const int base = from - u.tile, to = u.nt - u.tile < share - from ? base + u.nt : share;
    const Regions rg = regions_of(u.L, a.ns, a.nl);
    const size_t unit = (size_t)u.b * a.H + u.h;
    QFrag<NT> q;
    if (from > 0) load_queries<NT, AGG == SKV_AGG_MEAN>(queries(), a.Gi, x);
    make_queries<NG, NT, AGG == SKV_AGG_MEAN>(x, a.Gi, s_q, q);
    // the keys of this lane's rows: key, and 8 on
    int key = (rg.s_end & ~15) + (next - base) * 16 + g;
    float* out = a.scores + unit * (AGG == SKV_AGG_HEAD ? a.Gi : 1) * a.max_len + key;
#pragma unroll 1
    for (; next < to; next += W, key += 16 * W, out += 16 * W) {
      cp_async_wait<S - 2>();
      __syncwarp();
      feed.issue();
      float c[NT][4];
      logits<NG, NT>(ring + stage * kCell, q, c);
      const bool gone = feed.gone >> (S - 1) & 1u;
      stage = stage == S - 1 ? 0 : stage + 1;
      if constexpr (AGG == SKV_AGG_HEAD) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
          if (key + 8 * half >= rg.s_end && key + 8 * half < rg.l_start) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int head = 8 * nt + 2 * t + j;
                if (head < a.Gi)
                  out[(size_t)head * a.max_len + 8 * half] = gone ? NAN : c[nt][2 * half + j] * q.unit[nt][j];
              }
          }
      } else {
        float x[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (AGG == SKV_AGG_MAX) {
            x[half] = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (8 * nt + 2 * t + j < a.Gi) x[half] = max_nan(x[half], c[nt][2 * half + j] * q.unit[nt][j]);
            x[half] = max_nan(x[half], __shfl_xor_sync(0xffffffffu, x[half], 1));
            x[half] = max_nan(x[half], __shfl_xor_sync(0xffffffffu, x[half], 2));
          } else {  // columns 0 and 1, and 2 (3: none), in neighbouring lanes
            const float y = c[0][2 * half] + c[0][2 * half + 1];
            x[half] = (y + __shfl_xor_sync(0xffffffffu, y, 1)) * q.unit[0][0];
          }
        }
        // lane 0 of a quad writes the one key, lane 1 the other
        const int mine_key = key + 8 * t;
        if (t < 2 && mine_key >= rg.s_end && mine_key < rg.l_start) out[8 * t] = gone ? NAN : x[t & 1];
      }
    }
    from = to;
    if (from < share) {
      u.tile = u.nt;
      settle<kScore>(a, u);
    }
    __syncthreads();  // the queries' words have been read
  }
}

// ---------------------------------------------------------------------------- gather

// Eight codes (the bytes of a word, low half first) as pairs of bf16 values, the pair of a byte
// together: 128 + c by its bits, 136 off, and one fused product with the step and the centre
// (the first two bytes' word, the last two's).
__device__ __forceinline__ void values_of(uint32_t codes, uint32_t word01, uint32_t word23, uint32_t (&out)[4]) {
  const uint32_t lo = codes & 0x0f0f0f0fu, hi = codes >> 4 & 0x0f0f0f0fu, bias = 0x43084308u;
  const auto two = [](const uint32_t& x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c;  // (a selector's top bit: copies of a byte's sign, here 0)
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(c) : "r"(lo), "r"(hi), "r"(0x8480 + i * 0x101));
    c |= 0x43004300u;
    const uint32_t word = i < 2 ? word01 : word23, s = __byte_perm(word, word, 0x1010), z = __byte_perm(word, word, 0x3232);
    const __nv_bfloat162 v = __hfma2(__hsub2(two(c), two(bias)), two(s), two(z));
    out[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Four lanes a row: 16 bytes of codes each, four consecutive entries of every 16.  Finding a row is a
// step a round: its place's position, that one's entry, the row.  3,409 rows of K and V for 64 heads of requests
// of 32K: 52 MB read, 112 MB written, 28.5 us; what rows that lie alone leave of HBM's rate, and the 5 us
// until the first ones are found.
template <int NG, typename T>
__global__ void __launch_bounds__(256, 5) kv4_gather_kernel(const Kv4Args a, T* k_out, T* v_out, int n_att) {
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = lane & 3;
  const long long rows = (long long)a.B * a.H * n_att, stride = (long long)gridDim.x * 64;
  auto find = [&](long long r, Position& w) {
    w.t = -1;
    if (r >= rows) return;
    const long long unit = quotient(r, n_att);
    const int j = (int)(r - unit * n_att);
    Cursor c;
    c.b = (int)quotient(unit, a.H);
    c.h = (int)(unit - (long long)c.b * a.H);
    c.L = t == 0 && j == 0 && c.h == 0 ? load_len(a.seq_lens, c.b, a.max_len, a.status) : len_of(a, c.b);
    row_position(a, c, true, j, w);
  };
  const long long r0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 8 + (lane >> 2);
  Position position;
  Entry entry;
  find(r0, position);
  row_entry(a, t == 0, position, entry);
  find(r0 + stride, position);
  for (long long r = r0; r - (lane >> 2) < rows; r += stride) {  // (a warp's lanes together)
    const uint32_t at = row_id(a, t == 0, entry);
    const bool host = at >> 31;
    const size_t cell = (size_t)(at >> 4 & 0x7ffffffu) * kv4_cell(NG);
    const int rc = (int)(at & 15u);
    uint32_t codes[2][4], words[2][NG];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {  // both sides' loads together
#pragma unroll
      for (int i = 0; i < 4; ++i) codes[kv][i] = 0u;
#pragma unroll
      for (int i = 0; i < NG; ++i) words[kv][i] = 0u;
      if (at != kNoRow && (kv ? v_out : k_out) != nullptr) {
        const unsigned char* src =
            (const unsigned char*)(kv ? (host ? a.pool.host_v : a.pool.gpu_v) : (host ? a.pool.host_k : a.pool.gpu_k)) + cell;
        load_row<4>(src + rc * kCodeBytes + t * 16, codes[kv]);
        load_row<NG>(src + 16 * kCodeBytes + rc * 4 * NG, words[kv]);
      }
    }
    row_entry(a, t == 0, position, entry);
    find(r + 2 * stride, position);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      T* out = kv ? v_out : k_out;
      if (out == nullptr) continue;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {  // spans i .. i + 3
        const uint32_t b0 = codes[kv][i / 4], b1 = codes[kv][i / 4 + 2];  // their bytes: entries 4 t, + 1; + 2, + 3
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = words[kv][(i + k) * NG / 8];
            const float s = step_of(w), z = centre_of(w);
            auto value = [&](uint32_t b, int sh) {  // 2^23 + c by its bits (conversions are a quarter rate)
              return fmaf(s, __uint_as_float((b >> sh & 15u) | 0x4b000000u) - 8388616.f, z);
            };
            if (r < rows)
              *reinterpret_cast<float4*>(out + (size_t)r * kD + 16 * (i + k) + 4 * t) =
                  make_float4(value(b0, 8 * k), value(b0, 8 * k + 4), value(b1, 8 * k), value(b1, 8 * k + 4));
          }
        } else {
          uint32_t x[4], y[4];
          const uint32_t w01 = words[kv][i * NG / 8], w23 = words[kv][(i + 2) * NG / 8];
          values_of(b0, w01, w23, x);
          values_of(b1, w01, w23, y);
#pragma unroll
          for (int k = 0; k < 4; k += 2) {  // the even lane of a pair takes eight entries of span i + k, the odd lane of the next
            const uint32_t p0 = __shfl_xor_sync(0xffffffffu, t & 1 ? x[k] : x[k + 1], 1);
            const uint32_t p1 = __shfl_xor_sync(0xffffffffu, t & 1 ? y[k] : y[k + 1], 1);
            if (r < rows)
              *reinterpret_cast<uint4*>(out + (size_t)r * kD + 16 * (i + k) + (t & 1 ? 16 + 4 * (t - 1) : 4 * t)) =
                  t & 1 ? make_uint4(p0, p1, x[k + 1], y[k + 1]) : make_uint4(x[k], y[k], p0, p1);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- host

Kv4Args kv4_args(const skv_problem& p, const void* q, const PoolView& pool, const int32_t* idx, int32_t* status) {
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
  a.block_cells = (unsigned)((pool.per_head ? 1 : a.heads) * a.cells);
  a.n_gpu = (unsigned)pool.n_gpu;
  a.n_host = pool.host_k != nullptr ? (unsigned)pool.n_host : 0u;
  a.Gi = p.n_idx_q_heads / p.n_kv_heads;
  a.scale_log2 = (p.sm_scale > 0.f ? p.sm_scale : 1.f / sqrtf((float)p.d_qk)) * kLog2e;
  a.status = status;
  return a;
}

// CTAs for at most `units` units of `tiles` tiles
unsigned grid_of(long long units, long long tiles, int ctas) {
  long long n = (units * (tiles + kUnit) + kLeast - 1) / kLeast, most = (long long)num_sms() * ctas;
  if (most > kMaxParts) most = kMaxParts;
  n = n < most ? n : most;
  return (unsigned)(n < 1 ? 1 : n);
}

template <int NG, int NT, int MODE>
skv_status launch_attn(const Kv4Args& a, long long tiles, cudaStream_t st) {
  using Shape = AttnShape<NG, NT, MODE>;
  const auto kernel = kv4_attn_kernel<NG, NT, MODE>;
  const skv_status prep = prepare_kernel((const void*)kernel, Shape::kSmem);
  if (prep != SKV_OK) return prep;
  if (launch_dependent(kernel, dim3(grid_of((long long)a.B * a.H, tiles, Shape::kCtas)), dim3(32 * Shape::kW), Shape::kSmem, st, 1, a) !=
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
  constexpr int kSmem = kScoreW * kScoreStages * kv4_cell(NG);
  const skv_status prep = prepare_kernel((const void*)(wide ? kernel2 : kernel), kSmem);
  if (prep != SKV_OK) return prep;
  if (launch_dependent(wide ? kernel2 : kernel, dim3(grid_of((long long)a.B * a.H, tiles, kScoreCtas)), dim3(32 * kScoreW), kSmem, st, 1, a) != cudaSuccess)
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
  Kv4Args a = kv4_args(p, q, pool, idx, status);
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.ws = (float*)ws;
  a.desc = reinterpret_cast<int2*>((unsigned char*)ws + parts_bytes());
  const bool list = idx != nullptr;
  const long long n = list ? (long long)p.n_sink + p.topk + p.n_local : p.max_len;
  const long long tiles = (n + 15) / 16;
#define KV4_ATTN(NG)                                                                                            \
  (a.G > 8 ? (list ? launch_attn<NG, 2, kList>(a, tiles, st) : launch_attn<NG, 2, kDense>(a, tiles, st))        \
           : (list ? launch_attn<NG, 1, kList>(a, tiles, st) : launch_attn<NG, 1, kDense>(a, tiles, st)))
  return group == 32 ? KV4_ATTN(4) : group == 64 ? KV4_ATTN(2) : KV4_ATTN(1);
#undef KV4_ATTN
}

skv_status launch_kv4_score(const skv_problem& p, const void* q, const PoolView& pool, int group, float* scores,
                            int32_t* status, cudaStream_t st) {
  Kv4Args a = kv4_args(p, q, pool, nullptr, status);
  a.scores = scores;
  const long long tiles = ((long long)p.max_len + 15) / 16 + 1;
#define KV4_SCORE(NG)                                                                 \
  (p.group_agg == SKV_AGG_MEAN  ? launch_scores<NG, SKV_AGG_MEAN>(a, tiles, st)       \
   : p.group_agg == SKV_AGG_MAX ? launch_scores<NG, SKV_AGG_MAX>(a, tiles, st)        \
                                : launch_scores<NG, SKV_AGG_HEAD>(a, tiles, st))
  return group == 32 ? KV4_SCORE(4) : group == 64 ? KV4_SCORE(2) : KV4_SCORE(1);
#undef KV4_SCORE
}

skv_status launch_kv4_gather(const skv_problem& p, const PoolView& pool, int group, const int32_t* idx, void* k_out,
                             void* v_out, int32_t* status, cudaStream_t st) {
  const Kv4Args a = kv4_args(p, nullptr, pool, idx, status);
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
