// Attention of a batch over a shared prefix and every request's own tail.
//
//   out[b][j] = sum_{t < L_b} softmax(z)_t V_t,  z_t = sm_scale <q[b][j], K_t>
//
// The keys of the shared positions [0, P) are the same for every request, so the queries
// of all requests of a KV head -- row b * G + g of B * G rows -- meet them in matrix
// products on the tcgen05 tensor cores, and the prefix crosses HBM once; a tail [P, L_b)
// meets the G rows of its own request the same way.  Both are cut into tiles of 128 keys.
//
// prefix_attn_kernel, one persistent CTA an SM, 13 warps or 16:
//   warps 0-3, 4-7   softmax of slot 0 / slot 1 (a thread a query row)
//   warp 8           16 keys of a block of the GPU pool by one 4 KB TMA copy, into a ring of
//                    32 KB K / V stages in the 128-byte-swizzled layout that the MMA reads
//   warp 9, 13-15    every other key -- at a history's edge, in the host pool (over UVA), of
//                    blocks that 16 does not divide -- row by row, 16-byte cp.async with
//                    zeros for what is not attended (batch 8 on 32K keys all this way 48 us, by
//                    TMA 32); and the key masks
//   warp 10          cuts the CTA's share into segments, published in a ring for the other
//                    roles, and copies their query rows, by cp.async
//   warps 11, 12     issue the MMAs of slot 0 / slot 1 (converged, one elected lane: the
//                    operands' uniform registers then cost no per-lane serialisation, 100
//                    cycles an MMA otherwise; a warp a slot, so that one's bookkeeping runs
//                    under the other's MMAs)
// A *step* is one (128 query rows, 128 keys) tile: S = Q K^T (M128 N128, fp32 in TMEM),
// P = 2^(z - m) in bf16 over S's own columns, O += P V (A from TMEM, V read MN-major).
// Steps alternate between two slots of TMEM (S 128 + O 128 columns each), so that one
// slot's MMAs run under the other's softmax: with more than 128 rows the two slots hold
// two row tiles and share the keys; with up to 128 rows they take alternate key tiles.
// The running maximum is renewed only when it grows by more than 2^8 (P stays below 2^8
// relative to it, l and O in fp32 lose nothing), so O is rarely rescaled.
//
// Work is cut by key tiles: the CTAs form gangs (one member per pair of row tiles, so
// that members read the same keys at the same time) and gang c takes the tiles
// [c T / C, (c + 1) T / C) of all heads' prefixes; then come the tails' tiles, to the CTAs
// without prefix first, so that all have alike.  Each cut leaves every CTA that takes part a tile at least, so the segments
// of a unit -- runs of tiles of one head's prefix, or of one tail -- are those of
// consecutive CTAs.  A segment's O, m and l go to the workspace, at an index that grows
// with both the CTA and the unit, so no two segments share one and no atomics are needed.
// prefix_merge_kernel joins a row's partials by log-sum-exp, in a fixed order.
//
// What bounds it (8 KV heads of 8 query heads, CUDA graphs of 30 calls).  Few rows, long
// prefix -- batch 8 on 32K keys, 32.4 us: HBM while the prefix streams (134 MB, 20 us), then
// the tails, the start and the merge, a few us each.  Many rows -- batch 64 on 128K keys, 275
// GFLOP in 215 us, 1.28 PFLOP/s: the chain of a slot's step, 3,200 cycles.  The softmax takes
// 1,900 of them (the maximum 600, then 20 cycles a pair of keys, where a warp alone needs 12.5
// for the exponentials, sums and roundings without TMEM's latencies); the second half of P V
// and the next S 980 (S reads 8 KB of shared memory an MMA, 128 bytes a cycle of its 64: it
// runs a little below the pipe's rate); the hand-overs 330.  Both slots' MMAs together are
// 2,400, in turns; the tails of that case, 131 MB, take 22 us of it, near HBM's rate.  Small
// calls -- 4 requests on 777 keys, 10.6 us -- are a chain of first times: a role's first pass
// runs at some 25 cycles an instruction, so what lies on the way to the first S is short code.
// Instruction fetch was the bound of long calls, too: the roles run different code on the same
// SM, so loops are rolled, waits out of line, call sites single (unrolled over 64 keys the
// exponentials took 241 us in place of 226).
// Slower in the same measure: S of 64 keys at a time, twice buffered (233; an S as two N = 64
// MMAs costs more than one of N = 128, 234 by itself); sixteen softmax warps (244 against
// 226); P V begun after 96 of 128 keys (226) or in three parts (229); the first tile's maximum
// kept until a chunk of 32 keys outgrows it, without the pass for the maximum (236: the
// test and the maximum cost the exponentials' loop more than the pass did).
#include <cuda.h>  // CUtensorMap and its enums

#include "attn_common.cuh"
#include "tcgen05.cuh"

namespace skv {
namespace {

namespace px {
constexpr int kCtas = 152;             // one CTA an SM of a GB300 (a function of the problem alone: sizes the workspace)
constexpr int kRowWarps = 4;           // in place of one where rows come in bulk
constexpr int kTile = 128;             // keys a tile, query rows a tile
constexpr int kStageB = kTile * 256;   // a K, V or Q tile, 32 KB: [group of 8 rows][half of the dims][8 rows][128 bytes]
constexpr int kGroupB = 2048;          // a group of 8 rows
constexpr int kHalfB = 1024;           // one half of its dims
constexpr int kChunk = 16;             // keys of one TMA copy
constexpr int kChunks = kTile / kChunk;
constexpr int kRing = 5;               // K / V stages
constexpr int kQBufs = 2;
constexpr int kMasks = 8;              // key masks of the last tiles
constexpr int kSegs = 4;               // segments published ahead
constexpr int kSegReaders = 11;        // warps that read them: 8 softmax, TMA, 2 MMA; and the row warps
constexpr int kMaxGang = 4;            // pairs of row tiles that read the same keys together
constexpr float kGrow = 8.f;           // log2 growth of a row's maximum that renews it
constexpr uint32_t kTmemCols = 512;    // S0 S1 O0 O1, 128 columns each; P over the first 64 columns of S

// How the row tiles and the CTAs are arranged (host and device alike)
struct Plan {
  int rows, tiles, pairs, groups, gang, gangs;  // query rows, row tiles, pairs of them, groups of pairs, pairs a group
  int ntp;                                       // key tiles of the prefix
  int rp;                                        // rows of a prefix partial
  int each;                                      // what a CTA's share of the prefix counts in tail tiles, at most 2^20
};
__host__ __device__ inline Plan plan_of(int B, int H, int G, int P) {
  Plan pl;
  pl.rows = B * G;
  pl.tiles = (pl.rows + kTile - 1) / kTile;
  pl.pairs = (pl.tiles + 1) / 2;
  pl.groups = (pl.pairs + kMaxGang - 1) / kMaxGang;
  pl.gang = (pl.pairs + pl.groups - 1) / pl.groups;
  pl.ntp = (P + kTile - 1) / kTile;
  pl.gangs = kCtas / pl.gang;
  const long long tp = (long long)H * pl.groups * pl.ntp;
  // A gang has a tile at least (a unit's partials are then those of consecutive gangs), and more
  // than one before all CTAs are gangs: every gang of a unit leaves a partial a row, and CTAs
  // without prefix have the more of the tails.  79 x 4 tiles, 203 rows: one tile at least 33.2 us,
  // four 30.5, with tails of one key 22.0 and 20.7; 118 tiles: one 15.7 us, two 13.8, four 15.1;
  // 56 tiles: one 11.2, two 11.7, four 13.2.  A prefix without any tail loses by it: 29 requests
  // on 10,007 keys alone 21.6 us before the cut and 23.0 with it.
  const int most = pl.gangs, least = 2 * tp <= most ? 1 : tp <= most ? 2 : 4;
  if (tp < (long long)least * most) pl.gangs = (int)((tp + least - 1) / least);
  pl.rp = pl.rows < kTile ? pl.rows : kTile;
  const long long each = pl.gangs ? (tp + pl.gangs - 1) / pl.gangs * (pl.tiles > 1 ? 2 : 1) : 0;
  pl.each = (int)(each < 1 << 20 ? each : 1 << 20);
  return pl;
}

struct Args {
  const unsigned char* q;
  PoolView pool;
  const int32_t *ptable, *seq_lens;
  int B, H, Hq, G, P, max_len, bs;
  int tma;             // blocks are whole chunks of 16 keys
  int shift;           // log2 of the block size, -1: not a power of two
  float scale_log2;
  Plan pl;
  float *po, *pml;     // prefix partials: [(gang + unit) * members + member][row tile, if two][...]
  float *so, *sml;     // tail partials: [cta + unit][...]
  int *first, *last;   // [H * B]: the CTAs of a tail's first and last segment
  void* out;
  float* lse;
  int32_t* status;
};

// A tail's tiles start at the chunk of 16 that the prefix ends inside.
__host__ __device__ __forceinline__ int tail_base(int P) { return P & ~(kChunk - 1); }
// end of request b's tail (P: none, an empty request or one that ends inside the prefix), and its tiles
__device__ __forceinline__ int tail_end(const Args& a, int b) {
  int L = a.seq_lens[b];
  L = L > a.max_len ? a.max_len : L;
  return L > a.P ? L : a.P;
}
__device__ __forceinline__ int tail_tiles(const Args& a, int end) {
  return end > a.P ? (end - tail_base(a.P) + kTile - 1) / kTile : 0;
}

struct alignas(16) Seg {
  const int32_t* table;  // the positions' table row
  long long part;        // the partial's index
  int n;                 // key tiles; 0: the CTA's share is done
  int t0, lo, hi;        // first key position, the valid positions [lo, hi)
  int h, row0, n0, n1;   // KV head; first query row; live rows of the two row tiles (n1 = 0: one tile)
  int tail;              // a tail's segment, or the prefix's
};

// A CTA's segments in order (the walker warp's: every lane holds the same).
struct Walk {
  long long p0, p1;          // prefix tiles left: flattened (head, group, tile)
  long long srem;            // tail tiles left
  int scta;                  // the CTA's place among those with tail tiles
  int sh, sb, stile;         // the next tail tile
  int gang, member;          // the CTA's gang, its place in it
  bool scanned;
  __device__ __forceinline__ void init(const Args& a) {
    const Plan& pl = a.pl;
    gang = blockIdx.x;
    member = 0;
    if (pl.gang > 1) {
      gang = blockIdx.x / pl.gang;
      member = blockIdx.x - gang * pl.gang;
    }
    p0 = p1 = 0;
    if (gang < pl.gangs) {
      const long long tp = (long long)a.H * pl.groups * pl.ntp;
      p0 = gang * tp / pl.gangs;
      p1 = (gang + 1) * tp / pl.gangs;
    }
    srem = 0;
    scta = kCtas - 1 - (int)blockIdx.x;  // the last CTAs take the tails (the first the prefix, where there are few tiles)
    sh = sb = stile = 0;
    scanned = false;
  }
  // this CTA's range of the tails' tiles; its first tile by a scan of the requests' tile counts
  __device__ __forceinline__ void scan(const Args& a) {
    scanned = true;
    if (a.P >= a.max_len) return;
    const int lane = threadIdx.x & 31;
    const int per = (a.B + 31) / 32, b0 = lane * per < a.B ? lane * per : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
    long long mine = 0;
    int tails = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      const int n = tail_tiles(a, tail_end(a, b));
      mine += n;
      tails += n > 0;
    }
    long long at, lo;  // the first tile among one head's, the tiles before this lane's
    if (__all_sync(0xffffffffu, mine * a.H < 1 << 19)) {
      int incl = (int)mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const int total = __shfl_sync(0xffffffffu, incl, 31), ts = total * a.H;  // below 2^24
      // CTAs without tiles of the prefix, which stand first, take more: what makes all alike,
      // with a tile of two row tiles counted as two and a tail's start as one.  They have a
      // tile each before the others have any, so a unit's partials stay those of consecutive CTAs.
      const int with = a.pl.gangs * a.pl.gang, without = kCtas - with;
      int share = ts;
      if (with && ts > without) {
        const float starts = (float)(a.H * __reduce_add_sync(0xffffffffu, tails));
        share = (int)((float)ts * (1.f + (float)(with * a.pl.each) / ((float)ts + starts + 1.f)) *
                      ((float)without / (float)kCtas));
        share = share < without ? without : share > ts ? ts : share;
      }
      int place = scta, group = without, from = 0;
      if (place >= without) {
        from = share;
        share = ts - share;
        place -= without;
        group = with;
      }
      const int sn = share < group ? share : group;
      if (place >= sn) return;
      const uint32_t s0 = from + (uint32_t)place * (uint32_t)share / (uint32_t)sn;
      srem = from + (uint32_t)(place + 1) * (uint32_t)share / (uint32_t)sn - s0;
      sh = s0 / (uint32_t)total;
      at = s0 - (uint32_t)sh * total;
      lo = incl - (int)mine;
    } else {  // (so many tiles that the prefix's hardly count)
      long long incl = mine;
#pragma unroll 1
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const long long total = __shfl_sync(0xffffffffu, incl, 31), ts = total * a.H;
      const long long s0 = scta * ts / kCtas;
      srem = (scta + 1) * ts / kCtas - s0;
      sh = (int)(s0 / total);
      at = s0 - sh * total;
      lo = incl - mine;
    }
    int fb = 0, ft = 0;
    const bool here = at >= lo && at < lo + mine;
    if (here)
      for (int b = b0; b < b1; ++b) {
        const int n = tail_tiles(a, tail_end(a, b));
        if (at < lo + n) {
          fb = b;
          ft = (int)(at - lo);
          break;
        }
        lo += n;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    sb = __shfl_sync(0xffffffffu, fb, src);
    stile = __shfl_sync(0xffffffffu, ft, src);
  }
  // the next segment of the prefix, which is cut without a look at memory
  __device__ __forceinline__ bool next_prefix(const Args& a, Seg& s) {
    const Plan& pl = a.pl;
    while (p0 < p1) {
      const int up = (int)(p0 / pl.ntp), tile = (int)(p0 - (long long)up * pl.ntp);
      const long long left = p1 - p0;
      const int n = left < pl.ntp - tile ? (int)left : pl.ntp - tile;
      p0 += n;
      const int h = up / pl.groups, pair = (up - h * pl.groups) * pl.gang + member;
      if (pair >= pl.pairs) continue;  // the last group may be short of pairs
      const int r = pl.rows - pair * 2 * kTile;
      s.table = a.ptable;
      s.part = (long long)(gang + up) * pl.gang + member;
      s.n = n;
      s.t0 = tile * kTile;
      s.lo = 0;
      s.hi = a.P;
      s.h = h;
      s.row0 = pair * 2 * kTile;
      s.n0 = r < kTile ? r : kTile;
      s.n1 = r <= kTile ? 0 : (r - kTile < kTile ? r - kTile : kTile);
      s.tail = 0;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ void next(const Args& a, Seg& s) {
    if (next_prefix(a, s)) return;
    if (!scanned) scan(a);
    while (srem > 0) {
      const int end = tail_end(a, sb), nt = tail_tiles(a, end);
      if (stile >= nt) {
        stile = 0;
        if (++sb == a.B) {
          sb = 0;
          ++sh;
        }
        continue;
      }
      const int n = srem < nt - stile ? (int)srem : nt - stile, unit = sh * a.B + sb;
      if ((threadIdx.x & 31) == 0) {  // which CTAs hold the unit's partials
        if (stile == 0) a.first[unit] = scta;
        if (stile + n == nt) a.last[unit] = scta;
      }
      s.table = a.pool.table + (size_t)sb * a.pool.stride;
      s.part = (long long)scta + unit;
      s.n = n;
      s.t0 = tail_base(a.P) + stile * kTile;
      s.lo = a.P;
      s.hi = end;
      s.h = sh;
      s.row0 = sb * a.G;
      s.n0 = a.G;
      s.n1 = 0;
      s.tail = 1;
      stile += n;
      srem -= n;
      return;
    }
    s.n = 0;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(uint32_t x, uint32_t y, uint32_t z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)), "f"(__uint_as_float(z)));
  return r;
}
// two fp32 in one 64-bit register, and the packed operations on them
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// The ring's order of loads is that of their first use, so that each has about two tiles'
// time to land.  Two row tiles: K0 V0 K1 V1 ...  One: K0 K1 V0 K2 V1 ... -- S of step x + 2
// follows O of step x, so every V comes after the next tile's K, the segment's last one
// after the K of the segment behind it (after the last segment that place stays empty).
// A segment's places from its first one on, with `owed` = 1 where such a V comes into it:
__device__ __forceinline__ int k_place(bool two, int owed, int i) { return i == 0 ? 0 : owed + 2 * i - (two ? 0 : 1); }
__device__ __forceinline__ int v_place(bool two, int owed, int i) { return owed + 2 * i + (two ? 1 : 2); }
__device__ __forceinline__ int places(bool two, int owed, int n) { return owed + 2 * n - (two ? 0 : 1); }

// wait_or_abort with the spin out of line: the roles' loops stay small (instruction fetch
// is what the CTA's warps, at different places of the code, run short of first).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > 4000000000LL) {
      *abort = 1;
      if (status) atomicOr(status, SKV_DEV_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_slow(smem_u32(bar), parity, abort, status);
}

// full: two barriers a stage, of alternate rounds of the ring.  A slot's warp waits for the
// stages of its own steps only, so a stage may go through another round unseen by it; with
// one barrier the parity it waits for could be that of two rounds before.  With two, the
// round before on the same barrier (ten loads back) is over: the load that the warp saw
// last was issued after it had been handed back.
struct Bars {
  uint64_t seg[kSegs], seg_free[kSegs], full[2 * kRing], empty[kRing], qfull[kQBufs], qempty[kQBufs], mask[kMasks], s[2], p[2][2], o[2], x[2], turn[2], drain[2];
};

struct Shared {
  unsigned char buf[(kQBufs + kRing) * kStageB];  // first, on the 1 KB boundary of the swizzle
  float2 xml[2 * kTile];                          // the slots' (m, l) of a row
  uint4 masks[kMasks];
  Seg ring[kSegs];
  Bars bar;
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Shared) <= 232448, "227 KB a CTA");
constexpr int kSmem = (int)sizeof(Shared);

// A role's place in the published segments.  next() waits for one (false: the share is
// done, or the launch gives up); done() hands it back, once per warp.
struct Segs {
  const Args& a;
  Bars& bar;
  const Seg* ring;
  volatile int* abort;
  int k;
  __device__ __forceinline__ const Seg* next() {
    const int i = k % kSegs;
    bool ok = wait_on(&bar.seg[i], (uint32_t)(k / kSegs) & 1u, abort, a.status);
    if (__any_sync(0xffffffffu, !ok)) return nullptr;
    return ring[i].n > 0 ? &ring[i] : nullptr;
  }
  __device__ __forceinline__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.seg_free[k % kSegs]);
    ++k;
  }
};

// ---------------------------------------------------------------------------- gather warps
// Copies of single rows arrive on their barrier by themselves, a lane's when all it has
// issued have landed.  They are the generic proxy's writes: who waits on the barrier orders
// them before the MMA's reads by a proxy fence of its own.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
constexpr int kRowArrivals = 33;  // of a row warp on a stage: its lanes' copies, and what it stores
__device__ __forceinline__ void arrive_many(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(kRowArrivals) : "memory");
}

__device__ __forceinline__ int block_of(const Args& a, int t) { return a.shift >= 0 ? t >> a.shift : t / a.bs; }
__device__ __forceinline__ int in_block(const Args& a, int t) {
  return a.shift >= 0 ? t & (a.bs - 1) : t % a.bs;
}

// Reference of position t's row: its index in its pool, bit 62 for the host pool, -1 for none.
__device__ __forceinline__ long long row_ref(const Args& a, int h, int e, int t) {
  if (e >= 0) return e < a.pool.n_gpu ? ((long long)e * a.H + h) * a.bs + in_block(a, t) : -1;
  const long long hb = -(long long)e - 1;
  if (a.pool.host_k == nullptr || hb >= a.pool.n_host) return -1;
  return tc::kHostBit | ((hb * a.H + h) * a.bs + in_block(a, t));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 16 keys' rows of 256 bytes of a pool viewed as [rows / 8][2 halves][8 rows][64 dims]
__device__ __forceinline__ void tma_chunk(uint32_t dst, const CUtensorMap* map, int group, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(smem_u32(bar))
      : "memory");
}

// The chunks of four key tiles from t0 on, a lane each: the chunk's group of 8 rows in the
// GPU pool where a TMA copy takes it, else -1.
__device__ __forceinline__ int chunk_entry(const Args& a, const Seg* s, int t0, int lane) {
  const int t = t0 + kChunk * lane;
  return a.tma && t >= s->lo && t + kChunk <= s->hi ? s->table[block_of(a, t)] : -1;
}
__device__ __forceinline__ int chunk_group(const Args& a, int h, int e, int t0, int lane) {
  return e >= 0 && e < a.pool.n_gpu ? (e * a.H + h) * (a.bs >> 3) + (in_block(a, t0 + kChunk * lane) >> 3) : -1;
}

__device__ __forceinline__ void tma_role(const Args& a, const CUtensorMap* tk, const CUtensorMap* tv, Segs segs,
                                         Bars& bar, uint32_t base, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  if (a.tma && t5::elect_one()) {
    prefetch_map(tk);
    prefetch_map(tv);
  }
  pdl_wait();
  uint32_t sq = 0, par = 1;  // place in two rounds of the ring, parity of the stage's free phase
  int issued = 0;
  auto advance = [&] {
    ++issued;
    if (++sq == 2 * kRing) sq = 0;
    if (sq == 0 || sq == kRing) par ^= 1u;
  };
  // a stage of the chunks whose groups lanes 0-7 hold; false: the launch gives up
  auto load = [&](const CUtensorMap* map, int mine) {
    const uint32_t st = sq >= kRing ? sq - kRing : sq;
    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine >= 0) & 0xffu) * 2 * kGroupB;
    int group[kChunks];
#pragma unroll
    for (int v = 0; v < kChunks; ++v) group[v] = __shfl_sync(0xffffffffu, mine, v);
    const bool ok = wait_on(&bar.empty[st], par, abort, a.status);
    if (__any_sync(0xffffffffu, !ok)) return false;
    if (t5::elect_one()) {
      uint64_t* full = &bar.full[sq];
      const uint32_t dst = base + (kQBufs + st) * kStageB;
      if (bytes > 0)
        mbar_arrive_expect_tx(full, bytes);
      else
        mbar_arrive(full);
#pragma unroll
      for (int v = 0; v < kChunks; ++v)
        if (group[v] >= 0) tma_chunk(dst + v * 2 * kGroupB, map, group[v], full);
    }
    advance();
    return true;
  };
  int before = 0;           // groups of the tile whose V is owed
  bool owed = false, ok = true, more = true;
  while (ok && more) {
    const Seg* s = segs.next();
    more = s != nullptr;
    if (!more && (!owed || *abort)) break;
    // (behind the last segment one empty tile: its K's place stays empty, the V owed follows)
    const int n = more ? s->n : 1, h = more ? s->h : 0;
    const bool two = more && s->n1 > 0;
    int t0 = more ? s->t0 : 0, e = more ? chunk_entry(a, s, t0, lane) : -1, mine = -1;
    if (!more) advance();
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i, t0 += kTile) {
      if (more && (i & 3) == 0) {  // four tiles' entries at once, the next four already on their way
        mine = chunk_group(a, h, e, t0, lane);
        e = chunk_entry(a, s, t0 + 4 * kTile, lane);
      }
      const int now = __shfl_sync(0xffffffffu, mine, (8 * (i & 3) + lane) & 31);
      // this tile's K, a V that is owed, this tile's V with two row tiles
      const int loads = 1 + owed + two;
#pragma unroll 1
      for (int u = more ? 0 : 1; ok && u < loads; ++u) ok = load(u ? tv : tk, u == 1 && owed ? before : now);
      before = now;
      owed = !two;
    }
    if (more) segs.done();
  }
  if (!ok || *abort) {  // the launch gives up: copies in flight land (or their time runs out) before the memory goes
    for (int q = issued > kRing ? issued - kRing : 0; q < issued; ++q)
      mbar_wait_bounded(&bar.full[q % (2 * kRing)], (uint32_t)(q / (2 * kRing)) & 1u, 20000000LL);
  }
}

// Blocks of whole chunks of 16: a chunk's rows lie one behind another, 4 KB, so one table
// entry places them and a copy instruction takes two rows (four lines; half a row a lane
// would touch 32: batch 29's tails, with an entry a row, 38.2 us in place of 34.9).  Other
// block sizes: an entry a row.
// RW row warps, each takes every RW-th chunk of a load.
template <int RW>
__device__ __forceinline__ void rows_role(const Args& a, Segs segs, Bars& bar, unsigned char* gbase, uint4* masks,
                                          int part, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  bool ok = true;
  const bool chunked = a.bs % kChunk == 0;
  const int r16 = lane >> 1, half = lane & 1;    // other block sizes: a lane copies half a row
  const int odd = lane >> 4, piece = lane & 15;  // chunks: 16 lanes a row
  int T = 0;
  uint32_t sq = 0, par = 1;
  auto advance = [&] {
    if (++sq == 2 * kRing) sq = 0;
    if (sq == 0 || sq == kRing) par ^= 1u;
  };
  // lane l: rows l, l + 32, l + 64, l + 96 of this tile, of the tile whose V is owed; of
  // chunks, lanes 0-7 the first row (in [0]) and which of the 16 are attended
  long long ref[4], before[4];
  uint32_t bits = 0, bits_before = 0, whole_before = 0;
  bool owed = false, more = true;
  auto entry = [&](const Seg* s, int t) {  // of the chunk at t (0: none of it is attended)
    return chunked && t < s->hi && t + kChunk > s->lo ? s->table[block_of(a, t)] : 0;
  };
  while (ok && more) {
    const Seg* s = segs.next();
    more = s != nullptr;
    if (!more && (!owed || *abort)) break;
    const int n = more ? s->n : 1, h = more ? s->h : 0;
    const bool two = more && s->n1 > 0;
    int t0 = more ? s->t0 : 0, e = more ? entry(s, t0 + kChunk * lane) : 0;
    uint32_t all = 0, some = 0;  // four tiles' chunks: those that TMA takes; a lane each, the attended rows
    long long first = -1;        // and the first row
    if (!more) advance();
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i, ++T, t0 += kTile) {
      if (more && chunked) {
        if ((i & 3) == 0) {
          const int t = t0 + kChunk * lane, lo = s->lo - t, hi = s->hi - t;
          some = hi <= 0 || lo >= kChunk ? 0u : (hi >= kChunk ? 0xffffu : (1u << hi) - 1) & (lo > 0 ? ~0u << lo : ~0u);
          first = some ? row_ref(a, h, e, t) : -1;
          if (some && first < 0) {
            if (part == 0) flag(a.status, SKV_DEV_BAD_SLOT);
            some = 0;
          }
          all = __ballot_sync(0xffffffffu, a.tma && some == 0xffffu && !(first & tc::kHostBit));
          e = entry(s, t + 4 * kTile);
        }
        const int at = (8 * i + lane) & 31;
        ref[0] = __shfl_sync(0xffffffffu, first, at);
        bits = __shfl_sync(0xffffffffu, some, at);
      }
      const uint32_t whole = all & 0xffu;
      all >>= 8;
      uint32_t mask[4];
      if (more && !chunked) {
        int ent[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // all entries on their way at once
          const int t = t0 + 32 * j + lane;
          ent[j] = t >= s->lo && t < s->hi ? s->table[block_of(a, t)] : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + 32 * j + lane;
          const bool in = t >= s->lo && t < s->hi;
          ref[j] = in ? row_ref(a, h, ent[j], t) : -1;
          if (in && ref[j] < 0 && part == 0) flag(a.status, SKV_DEV_BAD_SLOT);
          mask[j] = __ballot_sync(0xffffffffu, ref[j] >= 0);
        }
      }
      // this tile's K, a V that is owed, this tile's V with two row tiles
      const int loads = 1 + owed + two;
#pragma unroll 1
      for (int u = more ? 0 : 1; ok && u < loads; ++u) {
        const bool old = u == 1 && owed;
        const uint32_t st = sq >= kRing ? sq - kRing : sq, w = old ? whole_before : whole;
        ok = wait_on(&bar.empty[st], par, abort, a.status);
        ok = !__any_sync(0xffffffffu, !ok);
        if (!ok) break;
        if (u == 0 && part == 0) {
          if (chunked && lane < 8)
            reinterpret_cast<uint16_t*>(masks + T % kMasks)[lane] = (uint16_t)bits;
          else if (!chunked && lane == 0)
            masks[T % kMasks] = make_uint4(mask[0], mask[1], mask[2], mask[3]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.mask[T % kMasks]);
        }
        if (w != 0xffu) {
          const unsigned char* gpu = (const unsigned char*)(u ? a.pool.gpu_v : a.pool.gpu_k);
          const unsigned char* host = (const unsigned char*)(u ? a.pool.host_v : a.pool.host_k);
          unsigned char* to = gbase + (kQBufs + st) * kStageB;
#pragma unroll 1
          for (int v = 0; v < kChunks; ++v, to += 2 * kGroupB) {
            if ((w >> v & 1u) || (v & (RW - 1)) != part) continue;
            if (chunked) {
              const long long r = __shfl_sync(0xffffffffu, old ? before[0] : ref[0], v);
              const uint32_t on = __shfl_sync(0xffffffffu, old ? bits_before : bits, v);
              if (on == 0u) {  // nothing attended: V zeros (S of these keys is masked whatever K is)
                if (u)
#pragma unroll
                  for (int k = 0; k < kChunk / 2; ++k)
                    *reinterpret_cast<uint4*>(to + k * 512 + lane * 16) = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              const unsigned char* src = ((r & tc::kHostBit) ? host : gpu) +
                                         (size_t)(r & tc::kRefRowMask) * tc::kRowBytes + lane * 16;
#pragma unroll
              for (int k = 0; k < kChunk / 2; ++k) {
                const int row = 2 * k + odd;
                const bool live = on >> row & 1u;
                tc::cp_async16_zfill(to + (piece >> 3) * kHalfB + (row >> 3) * kGroupB + (row & 7) * 128 +
                                         (((piece ^ row) & 7) << 4),
                                     live ? src + k * 2 * tc::kRowBytes : gpu, live);
              }
              continue;
            }
            const long long mine = old ? (v < 4 ? (v < 2 ? before[0] : before[1]) : (v < 6 ? before[2] : before[3]))
                                       : (v < 4 ? (v < 2 ? ref[0] : ref[1]) : (v < 6 ? ref[2] : ref[3]));
            const long long r = __shfl_sync(0xffffffffu, mine, 16 * (v & 1) + r16);
            const bool live = r >= 0;
            const unsigned char* src = live ? ((r & tc::kHostBit) ? host : gpu) +
                                                  (size_t)(r & tc::kRefRowMask) * tc::kRowBytes + half * 128
                                            : gpu;
            unsigned char* dst = to + (r16 >> 3) * kGroupB + half * kHalfB + (r16 & 7) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              tc::cp_async16_zfill(dst + ((c ^ (r16 & 7)) << 4), live ? src + c * 16 : src, live);
          }
          fence_proxy_async_smem();
          cp_async_arrive(&bar.full[sq]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.full[sq]);
        } else if (lane == 0) {
          arrive_many(&bar.full[sq]);
        }
        advance();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) before[j] = ref[j];
      bits_before = bits;
      whole_before = whole;
      owed = !two;
    }
    if (more) segs.done();
  }
  cp_async_commit();
  cp_async_wait<0>();  // (copies that no MMA waited for, where the launch gave up)
}

// ---------------------------------------------------------------------------- segments and query rows
__device__ __forceinline__ void walk_role(const Args& a, Bars& bar, Seg* ring, unsigned char* gbase,
                                          volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const int r16 = lane >> 1, half = lane & 1;
  const uint32_t row_off = (uint32_t)((r16 >> 3) * kGroupB + half * kHalfB + (r16 & 7) * 128);
  Walk walk;
  walk.init(a);
  auto publish = [&](const Seg& x, int k) {
    const bool ok = wait_on(&bar.seg_free[k % kSegs], (uint32_t)((k / kSegs) & 1) ^ 1u, abort, a.status);
    if (__any_sync(0xffffffffu, !ok)) return false;
    if (lane == 0) {
      ring[k % kSegs] = x;
      mbar_arrive(&bar.seg[k % kSegs]);
    }
    return true;
  };
  Seg s, s2;
  int nq = 0, k = 0;
  const bool early = walk.next_prefix(a, s);
  if (early && !publish(s, 0)) return;
  pdl_wait();
  if (!early) {
    walk.next(a, s);
    if (!publish(s, 0)) return;
  }
  while (s.n > 0) {
    for (int u = 0; u < (s.n1 > 0 ? 2 : 1); ++u, ++nq) {
      const int buf = nq & 1;
      const bool ok = wait_on(&bar.qempty[buf], (uint32_t)((nq >> 1) & 1) ^ 1u, abort, a.status);
      if (__any_sync(0xffffffffu, !ok)) {
        cp_async_commit();
        cp_async_wait<0>();
        return;
      }
      const int live = u ? s.n1 : s.n0;
#pragma unroll 1
      for (int v = 0; v * kChunk < live; ++v) {
        const int r = kChunk * v + r16;
        if (r < live) {
          const int row = s.row0 + u * kTile + r, b = row / a.G, gg = row - b * a.G;
          const unsigned char* src = a.q + (((size_t)b * a.Hq + (size_t)s.h * a.G + gg) * 2 + half) * 128;
          unsigned char* dst = gbase + buf * kStageB + v * 2 * kGroupB + row_off;
#pragma unroll
          for (int c = 0; c < 8; ++c) cp_async16(dst + ((c ^ (r16 & 7)) << 4), src + c * 16);
        }
      }
      cp_async_arrive(&bar.qfull[buf]);
    }
    walk.next(a, s2);
    if (!publish(s2, ++k)) break;
    s = s2;
  }
  cp_async_commit();
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------- MMA warp
// A step as its slot's issuing warp needs it, one word: ring stages and parities, the Q
// buffer, first and last uses.  Every stage and Q buffer is handed back by two arrivals,
// one of each slot, or both of one where the other does not use it.
namespace step {
constexpr uint32_t kSeq = 15u, kKPar = 4, kV = 5, kVPar = 9, kQBuf = 10, kQPar = 11;  // kSeq: place in two rounds
constexpr uint32_t kAlone = 1u << 12, kQAlone = 1u << 13, kFirst = 1u << 14, kLast = 1u << 15, kLive = 1u << 16;
}  // namespace step
// The slot's step words of a segment, 32 at a time: lane j holds the j-th of them.
struct Steps {
  Segs segs;
  int total, base, pos, cnt;  // steps of the segment, of which base are behind this batch; the batch's next and count
  int at, owed;               // the segment's first place in the ring, a V owed to it
  int nq, x;                  // Q buffers and steps (of both slots) before the segment
  int n, sub, slot;
  bool two, open;
  uint32_t words;
  __device__ __forceinline__ uint32_t next() {
    if (pos == cnt) {
      base += cnt;
      while (base == total) {  // a slot may have no step in a segment of one tile
        if (open) {
          at += places(two, owed, n);
          owed = two ? 0 : 1;
          nq += two ? 2 : 1;
          x += two ? 2 * n : n;
          segs.done();
        }
        const Seg* s = segs.next();
        open = s != nullptr;
        total = base = pos = cnt = 0;
        if (!open) return 0u;
        n = s->n;
        two = s->n1 > 0;
        sub = slot ^ (x & 1);
        total = two ? n : (n + 1 - sub) / 2;
      }
      cnt = total - base < 32 ? total - base : 32;
      pos = 0;
      const int j = base + (int)(threadIdx.x & 31);
      const int tile = two ? j : 2 * j + sub;
      const uint32_t k = (uint32_t)(at + k_place(two, owed, tile)), v = (uint32_t)(at + v_place(two, owed, tile));
      constexpr uint32_t kTwo = 2 * kRing;
      const uint32_t q = (uint32_t)(nq + (two ? sub : 0));
      uint32_t c = step::kLive | k % kTwo | ((k / kTwo) & 1u) << step::kKPar | (v % kTwo) << step::kV |
                   ((v / kTwo) & 1u) << step::kVPar | (q & 1u) << step::kQBuf | ((q >> 1) & 1u) << step::kQPar;
      if (!two) c |= step::kAlone;
      if (two || n == 1) c |= step::kQAlone;
      if (j == 0) c |= step::kFirst;
      if (j == total - 1) c |= step::kLast;
      words = c;
    }
    return __shfl_sync(0xffffffffu, words, pos++);
  }
};

__device__ __forceinline__ void mma_role(const Args& a, const Segs& segs, Bars& bar, uint32_t base, uint32_t tm,
                                         int slot, volatile int* abort) {
  const uint32_t id_s = t5::idesc_bf16(128, 128, false), id_o = t5::idesc_bf16(128, 128, true);
  // descriptors of buffer 0; a buffer is kStageB / 16 further in the address field
  const uint64_t dq = t5::desc_sw128(base, 16, kGroupB), dk = t5::desc_sw128(base + kQBufs * kStageB, 16, kGroupB);
  const uint64_t dv = t5::desc_sw128(base + kQBufs * kStageB, kHalfB, kGroupB);
  const uint32_t ts = tm + slot * 128, to = tm + 256 + slot * 128;
  Steps gen{segs, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, slot, false, false, 0u};
  pdl_wait();  // no bounded wait runs while the kernels before do
  bool ok = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok) ok = wait_on(b, parity, abort, a.status);
    ok = __all_sync(0xffffffffu, ok);
  };
  auto issue_s = [&](uint32_t c, bool k_there) {
    const uint32_t ksq = c & step::kSeq, ks = ksq >= kRing ? ksq - kRing : ksq, qb = (c >> step::kQBuf) & 1u;
    if (c & step::kFirst) wait(&bar.qfull[qb], (c >> step::kQPar) & 1u);
    if (!k_there) wait(&bar.full[ksq], (c >> step::kKPar) & 1u);
    if (!ok) return;
    fence_proxy_async_smem();
    t5::fence_after();
    const uint64_t qd = dq + qb * (kStageB >> 4), kd = dk + ks * (kStageB >> 4);
    if (t5::elect_one()) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {  // 16 of the 128 dims each
        const uint32_t off = ((uint32_t)(kk >> 2) * kHalfB + (kk & 3) * 32) >> 4;
        t5::mma(ts, qd + off, kd + off, id_s, kk > 0 ? 1u : 0u);
      }
      t5::commit(&bar.s[slot]);
      t5::commit(&bar.empty[ks]);
      if (c & step::kAlone) t5::commit(&bar.empty[ks]);
      if (c & step::kLast) {
        t5::commit(&bar.qempty[qb]);
        if (c & step::kQAlone) t5::commit(&bar.qempty[qb]);
      }
    }
  };
  // The slots' MMAs go in turns, O of a step and S of the next together: shared between the
  // slots, the pipe would finish both late and the softmaxes would run, and wait, in phase
  // (batch 64 on 128K keys, when they came: 230 us with turns, 262 without).
  auto pass_turn = [&] {
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.turn[slot ^ 1]);
  };
  auto issue_o = [&](uint32_t c, uint32_t p_par) {
    const uint32_t vsq = (c >> step::kV) & step::kSeq, vs = vsq >= kRing ? vsq - kRing : vsq;
    wait(&bar.full[vsq], (c >> step::kVPar) & 1u);
    fence_proxy_async_smem();
    const uint64_t vd = dv + vs * (kStageB >> 4);
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // 64 keys as soon as their P is there
      wait(&bar.p[slot][half], p_par);
      if (half == 0) wait(&bar.turn[slot], p_par ^ (slot ? 0u : 1u));
      if (!ok) return;
      t5::fence_after();
      if (t5::elect_one()) {
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)  // 16 of the 128 keys each
          t5::mma_ts(to, ts + kk * 8, vd + ((kk * 2 * kGroupB) >> 4), id_o,
                     kk > 0 ? 1u : ((c & step::kFirst) ? 0u : 1u));
        if (half) {
          t5::commit(&bar.empty[vs]);
          if (c & step::kAlone) t5::commit(&bar.empty[vs]);
          if (c & step::kLast) t5::commit(&bar.o[slot]);
        }
      }
    }
  };
  uint32_t now = 0u, p_par = 0u;
#pragma unroll 1
  while (ok) {  // O of a step, then S of the next one over its P
    const uint32_t nx = gen.next();
    if (!nx && !now) break;
    const bool there =
        nx && __all_sync(0xffffffffu, mbar_try_wait(&bar.full[nx & step::kSeq], (nx >> step::kKPar) & 1u));
    if (now) {
      issue_o(now, p_par);
      p_par ^= 1u;
      if (!there) pass_turn();  // nothing to follow yet: the other slot need not wait for it
    }
    if (ok && nx) issue_s(nx, there);
    if (now && there) pass_turn();
    now = nx;
  }
  // the operands in shared memory and TMEM outlive every MMA issued
  __syncwarp();
  if (t5::elect_one()) t5::commit(&bar.drain[slot]);
  mbar_wait_bounded(&bar.drain[slot], 0u);
}

// ---------------------------------------------------------------------------- softmax warps
__device__ __forceinline__ void softmax_role(const Args& a, Segs segs, Bars& bar, uint32_t tm, const uint4* masks, float2* xml,
                             volatile int* abort) {
  const int slot = threadIdx.x >> 7, wq = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  const uint32_t ts = tm + lanes + slot * 128, to = tm + lanes + 256 + slot * 128;
  pdl_wait();  // before the first partial: the workspace is the call before's until then
  int x = 0, T = 0, ns = 0, no = 0, nx = 0;
  bool ok = true;
  const Seg* sp;
  while (ok && (sp = segs.next()) != nullptr) {
    const Seg& s = *sp;
    const bool two = s.n1 > 0;
    const int sub = slot ^ (x & 1);
    const int mine = two ? s.n : (s.n + 1 - sub) / 2;
    const int live_rows = two && sub ? s.n1 : s.n0;
    const bool warp_live = wq * 32 < live_rows;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; ok && j < mine; ++j, ++ns) {
      const int tile = T + (two ? j : 2 * j + sub);
      ok = wait_on(&bar.mask[tile % kMasks], (uint32_t)(tile / kMasks) & 1u, abort, a.status);
      ok = ok && wait_on(&bar.s[slot], (uint32_t)ns & 1u, abort, a.status);
      ok = !__any_sync(0xffffffffu, !ok);
      if (!ok) break;
      t5::fence_after();
      if (warp_live) {
        const uint4 mk = masks[tile % kMasks];
        if ((mk.x & mk.y & mk.z & mk.w) != 0xffffffffu) {  // masked keys: -inf, in TMEM
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t v[32];
            t5::ld32(ts + c, v);
            const uint32_t mw = reinterpret_cast<const uint32_t*>(masks + tile % kMasks)[c >> 5];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((mw >> i) & 1u)) v[i] = 0xff800000u;
            t5::st32(ts + c, v);
          }
          t5::st_wait();
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        {
          uint32_t v[128];
#pragma unroll
          for (int c = 0; c < 128; c += 32) t5::ld32_async(ts + c, v + c);
#pragma unroll
          for (int c = 0; c < 128; c += 32) t5::ld_wait32(v + c);
#pragma unroll
          for (int i = 0; i < 128; i += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mx[u] = max3(__float_as_uint(mx[u]), v[i + u], v[i + 4 + u]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, row < live_rows && top > m + kGrow)) {
          // O of this slot is complete: S was issued after the last P V and committed after it.
          // A row's own maximum decides for it, so its bits do not depend on its neighbours.
          const bool grow = top > m + kGrow;
          const float f = grow ? ex2(m - top) : 1.f;
          m = grow ? top : m;
          l *= f;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            t5::ld32(to + ch * 32, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            t5::st32(to + ch * 32, o);
          }
        }
        const float mb = m == -INFINITY ? 0.f : -m;
        const uint64_t sc2 = pack2(a.scale_log2, a.scale_log2), mb2 = pack2(mb, mb);
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t v[32];
        t5::ld32_async(ts, v);
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t pk[16];
          t5::ld_wait32(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float z0, z1;
            unpack2(fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2, mb2), z0, z1);
            z0 = ex2(z0);
            z1 = ex2(z1);
            sum[i & 1] = add2(sum[i & 1], pack2(z0, z1));
            pk[i] = tc::pack_bf16(z0, z1);
          }
          t5::st16(ts + (c >> 1), pk);  // P of these keys, over S columns that have been read
          if (c < 96) t5::ld32_async(ts + c + 32, v);
          if (c == 32) {  // the first 64 keys' P V may start
            t5::st_wait();
            t5::fence_before();
            mbar_arrive(&bar.p[slot][0]);
          }
        }
        t5::st_wait();
        float l0, l1;
        unpack2(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
      } else {
        mbar_arrive(&bar.p[slot][0]);
      }
      t5::fence_before();
      mbar_arrive(&bar.p[slot][1]);
    }
    if (ok && mine > 0) {
      ok = wait_on(&bar.o[slot], (uint32_t)(no++) & 1u, abort, a.status);
      ok = !__any_sync(0xffffffffu, !ok);
      t5::fence_after();
    }
    if (l != l) m = NAN;  // a NaN key or query: the running maximum passes NaN over
    // the segment's partial, head-fastest in groups of 4 dims: [dim / 4][row][4]
    const int rp = s.tail ? a.G : a.pl.rp;
    const size_t at = (size_t)(s.tail ? s.part : 2 * s.part + (two ? sub : 0)) * rp;
    float* po = (s.tail ? a.so : a.po) + at * kD;
    float* ml = (s.tail ? a.sml : a.pml) + at * 2;
    if (two || s.n == 1) {  // the slot's own
      if (ok && warp_live && mine > 0) {
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t o[32];
          t5::ld32(to + ch * 32, o);
          if (row < live_rows)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(po + ((size_t)(ch * 8 + i) * rp + row) * 4) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if (row < live_rows) {
          ml[row] = m;
          ml[rp + row] = l;
        }
      }
    } else {
      // the slots took alternate tiles of the same rows: each joins half of the dims of both
      // (a row's TMEM lane is the same for the two slots' warps)
      xml[slot * kTile + row] = make_float2(m, l);
      mbar_arrive(&bar.x[0]);
      ok = ok && wait_on(&bar.x[0], (uint32_t)nx & 1u, abort, a.status);
      ok = !__any_sync(0xffffffffu, !ok);
      if (ok && warp_live) {
        t5::fence_after();
        const float2 m0 = xml[row], m1 = xml[kTile + row];
        const float mm = m0.x != m0.x || m1.x != m1.x ? NAN : fmaxf(m0.x, m1.x);
        const float w0 = m0.x == -INFINITY ? 0.f : ex2(m0.x - mm), w1 = m1.x == -INFINITY ? 0.f : ex2(m1.x - mm);
#pragma unroll 1
        for (int ch = 2 * slot; ch < 2 * slot + 2; ++ch) {
          uint32_t o[32], o1[32];
          t5::ld32(tm + lanes + 256 + ch * 32, o);
          t5::ld32(tm + lanes + 384 + ch * 32, o1);
          if (row < live_rows)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float c[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                c[u] = w0 * __uint_as_float(o[4 * i + u]) + w1 * __uint_as_float(o1[4 * i + u]);
              *reinterpret_cast<float4*>(po + ((size_t)(ch * 8 + i) * rp + row) * 4) = make_float4(c[0], c[1], c[2], c[3]);
            }
        }
        if (slot == 0 && row < live_rows) {
          ml[row] = mm;
          ml[rp + row] = w0 * m0.y + w1 * m1.y;
        }
      }
      // neither slot's O is overwritten before both have read it
      t5::fence_before();
      mbar_arrive(&bar.x[1]);
      ok = ok && wait_on(&bar.x[1], (uint32_t)(nx++) & 1u, abort, a.status);
      ok = !__any_sync(0xffffffffu, !ok);
    }
    x += two ? 2 * s.n : s.n;
    T += s.n;
    segs.done();
  }
}

template <int RW>
__global__ void __launch_bounds__(384 + 32 * RW, 1) prefix_attn_kernel(const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const Args a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  Bars& bar = sh.bar;
  const int t = threadIdx.x, warp = t >> 5;
  const uint32_t base = smem_u32(smem);
  if (base & 1023u) {  // the swizzle counts address bits from a 1 KB boundary
    flag(a.status, SKV_DEV_TIMEOUT);
    return;
  }
  if (t == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bar.seg[i], 1);
      mbar_init(&bar.seg_free[i], kSegReaders + RW);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.full[i], 1 + RW * kRowArrivals);
      mbar_init(&bar.full[kRing + i], 1 + RW * kRowArrivals);
      mbar_init(&bar.empty[i], 2);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(&bar.qfull[i], 32);
      mbar_init(&bar.qempty[i], 2);
    }
    for (int i = 0; i < kMasks; ++i) mbar_init(&bar.mask[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s[i], 1);
      mbar_init(&bar.p[i][0], 128);
      mbar_init(&bar.p[i][1], 128);
      mbar_init(&bar.o[i], 1);
      mbar_init(&bar.x[i], 256);
      mbar_init(&bar.turn[i], 1);
      mbar_init(&bar.drain[i], 1);
    }
    fence_barrier_init();
    sh.abort = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  pdl_release();  // every role that touches global memory waits for the kernels before by itself
  const uint32_t tm = sh.tmem;
  const Segs segs{a, bar, sh.ring, &sh.abort, 0};
  if (warp < 8) {
    softmax_role(a, segs, bar, tm, sh.masks, sh.xml, &sh.abort);
  } else {
    if (warp == 8)
      tma_role(a, &tk, &tv, segs, bar, base, &sh.abort);
    else if (warp == 9 || warp >= 13)
      rows_role<RW>(a, segs, bar, smem, sh.masks, RW == 1 || warp == 9 ? 0 : warp - 12, &sh.abort);
    else if (warp == 10)
      walk_role(a, bar, sh.ring, smem, &sh.abort);
    else
      mma_role(a, segs, bar, base, tm, warp - 11, &sh.abort);
  }
  t5::fence_before();
  __syncthreads();
  if (warp == 0) {
    t5::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmemCols) : "memory");
  }
}

// Joins the partials of 32 query rows of one KV head, kMergeDims of the 128 dims a CTA:
// lane = row, warp = (4 dims, one of PARTS shares of the partials), so every load of a
// partial is a coalesced float4.  A thread runs once over its share with a running maximum,
// kMergeBatch partials' loads in flight at a time (bound by their latency: one round for
// most shapes); the shares are joined through shared memory.  The order is fixed.  Four
// shares where the rows are few, two where the CTAs fill the device without (batch 8 on 32K
// keys in all 32.6 us with four, 33.8 with two; batch 64 on 128K 224 and 215).
constexpr int kMergeDims = 8;
constexpr int kMergeBatch = 5;

struct Joined {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float mp, float lp, float4 v) {
    if (mp == -INFINITY) return;  // an empty partial: its O was never written
    const float mn = mp != mp ? mp : fmaxf(m, mp);  // NaN stays: m, or the weights from then on
    const float f = m == -INFINITY ? 0.f : ex2(m - mn), w = ex2(mp - mn);
    m = mn;
    l = fmaf(w, lp, l * f);
    o.x = fmaf(w, v.x, o.x * f);
    o.y = fmaf(w, v.y, o.y * f);
    o.z = fmaf(w, v.z, o.z * f);
    o.w = fmaf(w, v.w, o.w * f);
  }
};

template <int PARTS>
__global__ void __launch_bounds__(PARTS * kMergeDims * 8, 8 / PARTS) prefix_merge_kernel(const Args a) {
  constexpr int kMergeWarps = PARTS * kMergeDims / 4;
  __shared__ float4 s_o[kMergeWarps][32];
  __shared__ float2 s_ml[kMergeWarps][32];
  pdl_release();
  const Plan& pl = a.pl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (pl.rows + 31) / 32;
  const int h = blockIdx.x / blocks, row = (blockIdx.x - h * blocks) * 32 + lane;
  const bool live = row < pl.rows;
  const int b = live ? row / a.G : 0, g = row - b * a.G;
  // the prefix's partials of this row: gangs c0 .. of its unit
  const int pair = row / (2 * kTile), pg = pair / pl.gang, member = pair - pg * pl.gang;
  const int up = h * pl.groups + pg;
  const bool two = pl.rows - pair * 2 * kTile > kTile;
  const int r_in = row & (kTile - 1);
  const long long tp = (long long)a.H * pl.groups * pl.ntp, u0 = (long long)up * pl.ntp;
  int c0 = 0, np = 0;
  if (pl.ntp > 0) {
    c0 = (int)(((u0 + 1) * pl.gangs - 1) / tp);
    np = (int)(((u0 + pl.ntp) * pl.gangs - 1) / tp) - c0 + 1;
  }
  const long long first_p = 2 * ((long long)(c0 + up) * pl.gang + member) + (two ? (row / kTile) & 1 : 0);
  const int step_p = 2 * pl.gang;
  const int part = warp / (kMergeDims / 4), d4 = blockIdx.y * (kMergeDims / 4) + warp % (kMergeDims / 4);
  const float* po = a.po + first_p * pl.rp * kD + ((size_t)d4 * pl.rp + r_in) * 4;
  const float* pml = a.pml + first_p * pl.rp * 2 + r_in;
  const int unit = h * a.B + b;
  pdl_wait();
  int L = live ? a.seq_lens[b] : 0;
  const int f = a.first[unit], e = a.last[unit];  // of no meaning without a tail
  Joined j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  float mp[kMergeBatch], lp[kMergeBatch];
  float4 v[kMergeBatch];
  auto fetch = [&](int i) {
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) {
      const int k = i + u * PARTS;
      mp[u] = -INFINITY;
      if (k < np && live) {
        const size_t at = (size_t)(k * step_p) * pl.rp;
        mp[u] = pml[at * 2];
        lp[u] = pml[at * 2 + pl.rp];
        v[u] = *reinterpret_cast<const float4*>(po + at * kD);
      }
    }
  };
  fetch(part);
  // the tail's partials: e - f + 1 consecutive ones of its unit; the first of this share flies
  // with the prefix's
  if (L < 0 || L > a.max_len || (L > 0 && L < a.P)) {
    if (blockIdx.y == 0 && warp == 0) flag(a.status, SKV_DEV_BAD_LENGTH);
    L = L > a.max_len ? a.max_len : 0;
  }
  const bool tail = L > a.P && f >= 0 && e < kCtas && f <= e;  // (else never written: an aborted launch)
  const int nt = tail ? e - f + 1 : 0;
  const size_t t_at = tail ? (size_t)((long long)f + unit) * a.G : 0;
  const float* so = a.so + t_at * kD + ((size_t)d4 * a.G + g) * 4;
  const float* sml = a.sml + t_at * 2 + g;
  float tm = -INFINITY, tl = 0.f;
  float4 to = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch_tail = [&](int i) {
    tm = -INFINITY;
    if (i < nt) {
      const size_t k = (size_t)i * a.G;
      tm = sml[k * 2];
      tl = sml[k * 2 + a.G];
      to = *reinterpret_cast<const float4*>(so + k * kD);
    }
  };
  fetch_tail(part);
#pragma unroll
  for (int u = 0; u < kMergeBatch; ++u) j.add(mp[u], lp[u], v[u]);
  for (int i = part + PARTS * kMergeBatch; i < np; i += PARTS * kMergeBatch) {
    fetch(i);
#pragma unroll
    for (int u = 0; u < kMergeBatch; ++u) j.add(mp[u], lp[u], v[u]);
  }
  j.add(tm, tl, to);
  for (int i = part + PARTS; i < nt; i += PARTS) {
    fetch_tail(i);
    j.add(tm, tl, to);
  }
  s_o[warp][lane] = j.o;
  s_ml[warp][lane] = make_float2(j.m, j.l);
  __syncthreads();
  if (part > 0 || !live) return;
#pragma unroll
  for (int i = 1; i < PARTS; ++i) {
    const int from = i * (kMergeDims / 4) + warp;
    const float2 ml = s_ml[from][lane];
    j.add(ml.x, ml.y, s_o[from][lane]);
  }
  const bool on = L > 0;
  // NaN stays NaN; an empty request, or no key at all: 0
  const float inv = on && (j.l > 0.f || j.l != j.l) ? 1.f / j.l : 0.f;
  const size_t hq = (size_t)b * a.Hq + (size_t)h * a.G + g;
  uint2 r = make_uint2(0u, 0u);
  if (on && inv != 0.f) {
    r.x = tc::pack_bf16(j.o.x * inv, j.o.y * inv);
    r.y = tc::pack_bf16(j.o.z * inv, j.o.w * inv);
  }
  *reinterpret_cast<uint2*>((__nv_bfloat16*)a.out + hq * kD + d4 * 4) = r;
  if (a.lse && d4 == 0) a.lse[hq] = on && (j.l > 0.f || j.l != j.l) ? kLn2 * (j.m + log2f(j.l)) : -INFINITY;
}

// A pool's K or V rows as [rows / 8][2 halves of the dims][8 rows][64 dims], in boxes of 16
// rows: one copy lands in the layout the MMA reads.
bool encode_pool(CUtensorMap* map, const void* ptr, long long rows) {
  const cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)(rows / 8)};
  const cuuint64_t strides[3] = {256, 128, 2048};
  const cuuint32_t box[4] = {64, 8, 2, 2};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn != nullptr && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  size_t po, pml, so, sml, first, last, total;
};
Layout layout_of(const skv_problem& p, int P) {
  const int G = p.n_q_heads / p.n_kv_heads;
  const Plan pl = plan_of(p.batch, p.n_kv_heads, G, P);
  const size_t units = (size_t)p.n_kv_heads * p.batch;
  const size_t pp = pl.ntp > 0 ? 2 * (size_t)(pl.gangs + (size_t)p.n_kv_heads * pl.groups) * pl.gang * pl.rp : 0;
  const size_t sp = P < p.max_len ? (kCtas + units) * G : 0;
  Layout l;
  l.po = 0;
  l.pml = l.po + align256(pp * kD * 4);
  l.so = l.pml + align256(pp * 2 * 4);
  l.sml = l.so + align256(sp * kD * 4);
  l.first = l.sml + align256(sp * 2 * 4);
  l.last = l.first + align256(units * 4);
  l.total = l.last + align256(units * 4);
  return l;
}

}  // namespace px
}  // namespace

size_t prefix_workspace_bytes(const skv_problem& p, int prefix_len) { return px::layout_of(p, prefix_len).total; }

skv_status launch_prefix_attn(const skv_problem& p, const void* q, const PoolView& pool, const skv_prefix& prefix,
                              void* out, float* lse, void* ws, int32_t* status, cudaStream_t st) {
  using namespace px;
  const int G = p.n_q_heads / p.n_kv_heads;
  const Layout lay = layout_of(p, prefix.len);
  unsigned char* w = (unsigned char*)ws;
  Args a;
  a.q = (const unsigned char*)q;
  a.pool = pool;
  a.ptable = prefix.table;
  a.seq_lens = p.seq_lens;
  a.B = p.batch;
  a.H = p.n_kv_heads;
  a.Hq = p.n_q_heads;
  a.G = G;
  a.P = prefix.len;
  a.max_len = p.max_len;
  a.bs = p.block_size;
  a.scale_log2 = (p.sm_scale > 0.f ? p.sm_scale : 1.f / sqrtf((float)p.d_qk)) * kLog2e;
  a.pl = plan_of(p.batch, p.n_kv_heads, G, prefix.len);
  a.po = (float*)(w + lay.po);
  a.pml = (float*)(w + lay.pml);
  a.so = (float*)(w + lay.so);
  a.sml = (float*)(w + lay.sml);
  a.first = (int*)(w + lay.first);
  a.last = (int*)(w + lay.last);
  a.out = out;
  a.lse = lse;
  a.status = status;
  CUtensorMap tk, tv;
  const long long rows = pool.n_gpu * p.n_kv_heads * p.block_size;
  a.shift = -1;
  for (int i = 0; i < 31; ++i)
    if (p.block_size == 1 << i) a.shift = i;
  a.tma = p.block_size % kChunk == 0 && rows > 0 && rows / 8 < (1LL << 31);
  if (a.tma && (!encode_pool(&tk, pool.gpu_k, rows) || !encode_pool(&tv, pool.gpu_v, rows))) return SKV_ERR_CUDA;
  // Four row warps where whole histories are theirs -- blocks that 16 does not divide, a host
  // pool -- and one where they have the histories' ends alone: batch 8 on 32K keys, every key by
  // rows, 47.8 us with four and 77.7 with one; batch 64 on 128K by TMA 219 with four, 215 with one.
  const bool bulk = p.block_size % kChunk != 0 || pool.host_k != nullptr;
  const auto kernel = bulk ? prefix_attn_kernel<kRowWarps> : prefix_attn_kernel<1>;
  const skv_status prep = prepare_kernel((const void*)kernel, px::kSmem);
  if (prep != SKV_OK) return prep;
  if (launch_dependent(kernel, dim3(kCtas), dim3(384 + 32 * (bulk ? kRowWarps : 1)), px::kSmem, st, 1, tk, tv, a) !=
      cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  const long long blocks = (long long)((a.pl.rows + 31) / 32) * a.H;
  const bool few = blocks * (kD / kMergeDims) <= 2 * kCtas;
  if (launch_dependent(few ? prefix_merge_kernel<4> : prefix_merge_kernel<2>, dim3((unsigned)blocks, kD / kMergeDims),
                       dim3((few ? 4 : 2) * kMergeDims * 8), 0, st, 1, a) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

}  // namespace skv
