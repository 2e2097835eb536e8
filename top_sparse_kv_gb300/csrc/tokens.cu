// New tokens: per-head RMS norm and rotation of queries and keys in one pass over their
// rows, and the append of K and V rows to the paged pool through the slot table.
//
//   norm      y_j = gamma_j x_j / sqrt(mean_{i < norm_dim} x_i^2 + eps)
//   rotation  (a, b) -> (a cos - b sin, b cos + a sin) at the angle t * inv_freq[i]
//
// Each row is read once and written once.  A CTA takes a token (or a part of its rows) at a
// time: its cosines and sines are computed once into shared memory and the warps walk the
// rows of its heads -- queries, keys, values -- a row spread over lanes in 16-byte vectors,
// so loads and stores are whole 16-byte accesses of consecutive lanes and the sum of squares
// is a butterfly over the row's lanes.
//
// With everything computed per row this is bound by instruction issue before it is by HBM
// (8,192 tokens of 72 rows of 128 bf16, 302 MB: 103 us), so what does not change from row to
// row comes once a token: with g the weights an entry becomes f (x A + x' B), A = g cos,
// B = -+ g' sin, x' its partner and f the row's 1 / rms.  Now 53.7 us, 5.6 TB/s, 0.83 of the
// copy rate, at 66 % of the issue slots; 8 tokens are a launch, 3.6 us in a graph.
#include "kv4.cuh"

namespace skv {
namespace {

constexpr int kLongWarps = 4;

struct TokenArgs {
  const unsigned char *q, *k, *v;
  long long qs, ks, vs;  // bytes from token to token
  unsigned char *q_out, *k_out;
  long long qos, kos;
  PoolView pool;  // append: the pool rows take K and V
  const int32_t *positions, *requests, *seq_lens;
  int n_tokens, B, H, Hq, d, dv, max_len, bs;
  int rot_start, rot_dim, style, norm_dim;
  float eps, inv_norm;
  const float* inv_freq;
  const unsigned char *gq, *gk;
  int32_t* status;
  int parts;  // CTAs a token
  int stage;  // bytes of a staged item's rows
};

// cos and sin of t * f: the turn t f / 2 pi as a 64-bit fraction, whose integer product
// with t wraps modulo one turn by itself.  One position's turn is f times 1 / 2 pi in two
// parts, the large one's product exact by its remainder and put into place by its bits (fp64
// instructions are scarce: four here); it is off by less than 2 * 2^-64 for |f| to 2^14, and
// t's by less than 2^-32 wherever t lies.  (With one double f / 2 pi carries 2^-53 of itself,
// times t: at t = 2^31 four parts in 2^24 of a turn for f = 6.)  The nearest quarter turn
// comes off in integers too; what is left is at most an eighth of a turn, so its fp32
// rounding is at most 2^-25 of pi / 4.
__device__ __forceinline__ unsigned long long turn_of(float f) {  // one position's turn, of 2^64
  constexpr double kHi = 0.15915494309189535;  // 1 / 2 pi, and what it lacks
  constexpr float kLo = -9.8393382e-18f;
  const double hi = (double)f * kHi;
  const float lo = fmaf(f, kLo, (float)fma((double)f, kHi, -hi));
  const long long b = __double_as_longlong(hi);
  const int up = (int)((b >> 52) & 0x7ff) - 1075 + 64;  // from the mantissa's last place to 2^-64
  unsigned long long turn = (unsigned long long)((b & ((1ll << 52) - 1)) | (1ll << 52));
  turn = up >= 0 ? (up < 64 ? turn << up : 0ull) : (up > -64 ? turn >> -up : 0ull);
  return (b < 0 ? 0ull - turn : turn) + (unsigned long long)__float2ll_rn(lo * 18446744073709551616.f);
}
__device__ __forceinline__ float2 cos_sin_of(unsigned long long ph) {
  const unsigned long long near = ph + (1ull << 61);
  const int quarter = (int)(near >> 62);
  const long long rem = (long long)(near & ((1ull << 62) - 1)) - (1ll << 61);
  float s, c;
  sincospif((float)(int)(rem >> 30) * 1.16415321826934814453e-10f, &s, &c);  // 2^-33: half turns
  const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -cc : cc, quarter >= 2 ? -ss : ss);
}
__device__ __forceinline__ float2 turn_cos_sin(int t, float f) {
  return cos_sin_of(turn_of(f) * (unsigned long long)t);
}

// What a CTA's token needs once: its request, position and, for an append, the pool rows of
// KV head 0 (null: none) and the bytes from head to head.
struct Token {
  int req, pos;
  bool live;
  unsigned char *k, *v;
  size_t k_head, v_head;
};

__device__ __forceinline__ Token token_of(const TokenArgs& a, int tok, bool reports) {
  Token t;
  t.live = false;
  t.req = a.requests ? a.requests[tok] : tok;
  t.pos = -1;
  t.k = t.v = nullptr;
  t.k_head = t.v_head = 0;
  if (a.requests && t.req < 0) return t;
  const bool needs_req = a.pool.table != nullptr || a.positions == nullptr || a.requests != nullptr;
  if (needs_req && t.req >= a.B) {
    // (a negative position: padding, whatever its request)
    if (reports && (a.positions == nullptr || a.positions[tok] >= 0)) flag(a.status, SKV_DEV_BAD_INDEX);
    return t;
  }
  t.pos = a.positions ? a.positions[tok] : a.seq_lens[t.req] - 1;
  if (t.pos < 0 || t.pos >= a.max_len) {
    const bool bad = a.positions ? t.pos >= 0 : (t.pos < -1 || t.pos >= a.max_len);
    if (bad && reports) flag(a.status, SKV_DEV_BAD_LENGTH);
    return t;
  }
  t.live = true;
  return t;
}

// The pool rows of the token in KV head h's blocks: row addresses, null for a bad entry.  NG > 0
// groups a row: of a pool in 4 bits, the addresses of the cells that hold them.
template <int NG = 0>
__device__ __forceinline__ void pool_rows(const TokenArgs& a, const Token& t, int h, int elem, unsigned char** k,
                                          unsigned char** v) {
  *k = *v = nullptr;
  const int e = table_row(a.pool, t.req, h, a.H)[t.pos / a.bs];
  const int off = t.pos % a.bs;
  const bool gpu = e >= 0;
  size_t row;
  if (gpu && e < a.pool.n_gpu) {
    row = gpu_block_row(a.pool, e, h, a.H, a.bs) + off;
  } else if (!gpu && a.pool.host_k != nullptr && -(long long)e - 1 < a.pool.n_host) {
    row = ((size_t)(-(long long)e - 1) * a.H + h) * a.bs + off;
  } else {
    flag(a.status, SKV_DEV_BAD_SLOT);
    return;
  }
  if constexpr (NG > 0) {
    const size_t at = row / kCellTokens * kv4_cell(NG);
    *k = (unsigned char*)(gpu ? a.pool.gpu_k : a.pool.host_k) + at;
    if (a.v) *v = (unsigned char*)(gpu ? a.pool.gpu_v : a.pool.host_v) + at;
  } else {
    *k = (unsigned char*)(gpu ? a.pool.gpu_k : a.pool.host_k) + row * a.d * elem;
    if (a.v) *v = (unsigned char*)(gpu ? a.pool.gpu_v : a.pool.host_v) + row * a.dv * elem;
  }
}

// Where row r of the token (queries, keys, values in order) comes from and goes to (null: nowhere).
template <int ELEM>
__device__ __forceinline__ const unsigned char* row_from(const TokenArgs& a, int tok, int r, int nq, int nk) {
  if (r < nq) return a.q + tok * a.qs + (size_t)r * a.d * ELEM;
  if (r < nq + nk) return a.k + tok * a.ks + (size_t)(r - nq) * a.d * ELEM;
  return a.v + tok * a.vs + (size_t)(r - nq - nk) * a.dv * ELEM;
}
template <int ELEM, int NG = 0>
__device__ __forceinline__ unsigned char* row_to(const TokenArgs& a, const Token& t, int tok, int r, int nq, int nk) {
  if (r < nq) return a.q_out + tok * a.qos + (size_t)r * a.d * ELEM;
  const bool is_v = r >= nq + nk;
  const int h = is_v ? r - nq - nk : r - nq;
  if (a.pool.table == nullptr) return a.k_out + tok * a.kos + (size_t)h * a.d * ELEM;
  if (a.pool.per_head) {
    unsigned char *k, *v;
    pool_rows<NG>(a, t, h, ELEM, &k, &v);
    return is_v ? v : k;
  }
  unsigned char* base = is_v ? t.v : t.k;
  return base ? base + h * (is_v ? t.v_head : t.k_head) : nullptr;
}

// One shared table entry serves every head: looked up once a token.
template <int ELEM, int NG = 0>
__device__ __forceinline__ void find_pool_rows(const TokenArgs& a, Token& t) {
  if (a.pool.table == nullptr || a.pool.per_head) return;
  pool_rows<NG>(a, t, 0, ELEM, &t.k, &t.v);
  t.k_head = NG ? (size_t)(a.bs / kCellTokens) * kv4_cell(NG) : (size_t)a.bs * a.d * ELEM;
  t.v_head = NG ? t.k_head : (size_t)a.bs * a.dv * ELEM;
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const float* x) {  // the one rounding
  constexpr int VE = Vec<T>::N;
  __align__(16) T out[VE];
#pragma unroll
  for (int j = 0; j < VE; ++j) out[j] = from_float<T>(x[j]);
  return *reinterpret_cast<uint4*>(out);
}

// A row of 128 entries into its cell, VE = 128 / LPR of them a lane.  The lane's bytes are its
// entries' pairs in order; the cell wants byte 8 i + u at 8 u + i, so lanes exchange bytes until
// each holds neighbours of one u: lanes whose i differs in a bit give each other the bytes whose u
// differs in the same bit.  Every lane of the row's LPR takes part; cell null: nothing is written.
// 8,192 tokens of 64 query, 8 key and 8 value heads of 128 bf16 go in 78 us, 323 MB, bound by issue (65 %
// of the slots; the query rows, norm and rotation alone, are most of it); 64 tokens in 5.  Codes come by a
// reciprocal, for steps under 2^-100 by a division an entry.  8,192 tokens of 8 query heads and one KV head, half
// a warp idle at every row: 48 us; 16 and two: 42.
template <int VE, int LPR, int NG>
__device__ __forceinline__ void put_row4(const float (&x)[VE], unsigned char* cell, int rc, int sub) {
  constexpr int kLanes = LPR / NG;  // of a group
  float lo = x[0], hi = x[0], s, z;
#pragma unroll
  for (int j = 1; j < VE; ++j) lo = min_nan(lo, x[j]), hi = max_nan(hi, x[j]);
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const uint32_t word = kv4_word(lo, hi, &s, &z);
  uint32_t w = 0;
  const float inv = 1.f / s;
#pragma unroll
  for (int j = 0; j < VE; ++j) w += kv4_code(x[j], s, z, inv) << (4 * j);
  // (a step of 0 among them; lanes without a row have one too, and no say)
  if (__any_sync(0xffffffffu, cell != nullptr && s < 0x1p-100f)) {
    w = 0;
#pragma unroll 1
    for (int j = VE - 1; j >= 0; --j) {
      float y = x[0];
#pragma unroll
      for (int i = 1; i < VE; ++i) y = j == i ? x[i] : y;
      w = w << 4 | kv4_code(y, s, z);
    }
  }
  if constexpr (VE == 8) {  // sub: u's bit 2, i's bits 0, 1, 2; the word: u's bits 0, 1
    uint32_t y = __shfl_xor_sync(0xffffffffu, w, 2);
    w = __byte_perm(w, y, sub & 2 ? 0x3715 : 0x6240);
    y = __shfl_xor_sync(0xffffffffu, w, 4);
    w = __byte_perm(w, y, sub & 4 ? 0x3276 : 0x5410);
    const int u = (sub & 1) * 4 + (sub >> 2 & 1) * 2 + (sub >> 1 & 1);
    if (cell != nullptr) *reinterpret_cast<uint32_t*>(cell + rc * kCodeBytes + 8 * u + 4 * (sub >> 3)) = w;
  } else {  // sub: u's bits 1, 2, i's bits 0, 1, 2; the half word: u's bit 0
    const uint32_t y = __shfl_xor_sync(0xffffffffu, w, 4);
    w = __byte_perm(w, y, sub & 4 ? 0x15 : 0x40);
    const int u = (sub & 3) * 2 + (sub >> 2 & 1);
    if (cell != nullptr)
      *reinterpret_cast<uint16_t*>(cell + rc * kCodeBytes + 8 * u + 4 * (sub >> 4) + 2 * (sub >> 3 & 1)) = (uint16_t)w;
  }
  if (cell != nullptr && sub % kLanes == 0)
    reinterpret_cast<uint32_t*>(cell + kCellTokens * kCodeBytes)[rc * NG + sub / kLanes] = word;
}

// Rows of at most LPR vectors: LPR lanes a row (a vector a lane), a token's rows staged in
// shared memory.  Persistent CTAs of W row warps and one that runs ahead: for every item --
// a token, or a part of its rows where tokens are few or its rows many --
// it fetches the rows by bulk copies (they are consecutive in memory), looks up the
// position and the pool rows and writes the coefficients A and B of queries and keys,
// kTokStages items deep, so the row warps meet no latency but shared memory's.  (A third
// stage bought nothing: 1,237 fp32 tokens 15.1 us with three, 13.8 with two.)
constexpr int kTokStages = 2;
constexpr int kTokStageMax = 40 * 1024;

struct StageInfo {
  Token t;
  int tok, r0, r1;  // the item's rows of the token
};
struct alignas(16) TokenBars {
  unsigned char zeros[16];  // the partner of entries that are not turned: -0, which adds to either zero nothing
  uint64_t full[kTokStages], empty[kTokStages];
  int abort;
};
constexpr int kInfoBytes = 128;
// Row warps and resident CTAs a SM: with half-warp rows (bf16) four warps share a token's
// fixed costs better than eight (8,192 tokens of 72 rows 54.0 us against 56.9), with whole-warp
// rows eight are better than four (1,237 fp32 tokens of 48 rows 13.6 against 16.4).
template <int LPR>
constexpr int kRowWarps = LPR == 16 ? 4 : 8;
template <int LPR>
constexpr int kTokCtas = LPR == 16 ? 4 : 3;
constexpr int kTokSmemMax = kInfoBytes + kTokStages * (kInfoBytes + 4096 + kTokStageMax);
static_assert(sizeof(StageInfo) <= kInfoBytes && sizeof(TokenBars) <= kInfoBytes, "");

// PAIR: partners are neighbours of the same vector, else `half` entries away.  PART: the norm
// covers a part of the row (as a test at run time it costs 5 % of every other call).  NG > 0: K and V
// rows go into a pool in 4 bits, NG groups a row.
template <typename T, int LPR, bool PAIR, bool PART, int NG>
__global__ void __launch_bounds__(32 * kRowWarps<LPR> + 32, kTokCtas<LPR>) token_rows_kernel(const TokenArgs a) {
  constexpr int W = kRowWarps<LPR>;
  constexpr int VE = Vec<T>::N, RPW = 32 / LPR, ELEM = sizeof(T);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long turns[LPR * VE / 2];  // of one position, an angle each
  TokenBars& bar = *reinterpret_cast<TokenBars*>(smem);
  const int half = a.rot_dim >> 1, d = a.d;
  const int stage_bytes = kInfoBytes + 16 * d + a.stage;  // info; A, B of queries, of keys; rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = a.q ? a.Hq : 0, nk = a.k ? a.H : 0, nv = a.v ? a.H : 0;
  const int rows = nq + nk + nv, per = (rows + a.parts - 1) / a.parts;
  const long long items = (long long)a.n_tokens * a.parts;
  const int rowb = d * ELEM, vrowb = a.dv * ELEM;
  volatile int* abort = &bar.abort;
  auto stage = [&](int s) { return smem + kInfoBytes + s * stage_bytes; };
  auto weight = [&](const unsigned char* g, int j) -> float {
    if (g == nullptr || j >= a.norm_dim) return 1.f;
    if constexpr (ELEM == 2)
      return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(g)[j] << 16);
    else
      return reinterpret_cast<const float*>(g)[j];
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTokStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], W);
    }
    fence_barrier_init();
    bar.abort = 0;
    constexpr uint32_t kNone = ELEM == 2 ? 0x80008000u : 0x80000000u;
    *reinterpret_cast<uint4*>(bar.zeros) = make_uint4(kNone, kNone, kNone, kNone);
  }
  pdl_release();
  pdl_wait();
  // entries that are not turned: A = g, B = 0 in every stage, for good (x g + 0 * -0 is x g, its zero's sign too)
  for (int i = threadIdx.x; i < 2 * d; i += 32 * W + 32) {
    const int k = i / d, j = i - k * d;
    const float g = weight(k ? a.gk : a.gq, j);
    for (int s = 0; s < kTokStages; ++s) {
      float* t = reinterpret_cast<float*>(stage(s) + kInfoBytes) + 2 * k * d;
      t[j] = g;
      t[d + j] = 0.f;
    }
  }
  for (int i = threadIdx.x; i < half; i += 32 * W + 32) turns[i] = turn_of(a.inv_freq[i]);
  __syncthreads();

  if (warp == W) {
    constexpr int kAngles = LPR * VE / 64;  // of a lane: half is at most LPR * VE / 2
    unsigned long long turn[kAngles];
    float g[kAngles][4];  // the weights of an angle's pair: queries, keys
    int at[kAngles][2];   // its entries
#pragma unroll
    for (int u = 0; u < kAngles; ++u) {
      const int i = lane + 32 * u;
      if (i < half) {
        turn[u] = turns[i];
        at[u][0] = a.rot_start + (PAIR ? 2 * i : i);
        at[u][1] = a.rot_start + (PAIR ? 2 * i + 1 : i + half);
#pragma unroll
        for (int k = 0; k < 4; ++k) g[u][k] = weight(k < 2 ? a.gq : a.gk, at[u][k & 1]);
      }
    }
    int n = 0;
    for (long long it = blockIdx.x; it < items; it += gridDim.x, ++n) {
      const int s = n % kTokStages;
      const bool ok = wait_or_abort(&bar.empty[s], (uint32_t)((n / kTokStages) & 1) ^ 1u, abort, a.status);
      if (__any_sync(0xffffffffu, !ok)) break;
      const int tok = (int)(it / a.parts), r0 = (int)(it - (long long)tok * a.parts) * per;
      const int r1 = r0 + per < rows ? r0 + per : rows;
      unsigned char* st = stage(s);
      float* co = reinterpret_cast<float*>(st + kInfoBytes);
      if (lane == 0) {  // the rows: consecutive ranges of q, k and v
        unsigned char* to = st + kInfoBytes + 16 * d;
        const int q0 = r0 < nq ? r0 : nq, q1 = r1 < nq ? r1 : nq;
        const int k0 = r0 > nq ? r0 - nq : 0, k1 = r1 > nq ? (r1 - nq < nk ? r1 - nq : nk) : 0;
        const int v0 = r0 > nq + nk ? r0 - nq - nk : 0, v1 = r1 > nq + nk ? r1 - nq - nk : 0;
        const uint32_t qb = q1 > q0 ? (q1 - q0) * rowb : 0, kb = k1 > k0 ? (k1 - k0) * rowb : 0;
        const uint32_t vb = v1 > v0 ? (v1 - v0) * vrowb : 0;
        mbar_expect_tx(&bar.full[s], qb + kb + vb);
        if (qb) bulk_g2s(to, a.q + tok * a.qs + (size_t)q0 * rowb, qb, &bar.full[s]);
        if (kb) bulk_g2s(to + qb, a.k + tok * a.ks + (size_t)k0 * rowb, kb, &bar.full[s]);
        if (vb) bulk_g2s(to + qb + kb, a.v + tok * a.vs + (size_t)v0 * vrowb, vb, &bar.full[s]);
      }
      Token t = token_of(a, tok, lane == 0 && r0 == 0);
      if (t.live) {
        find_pool_rows<ELEM, NG>(a, t);
#pragma unroll
        for (int u = 0; u < kAngles; ++u)
          if (lane + 32 * u < half) {
            const float2 c = cos_sin_of(turn[u] * (unsigned long long)t.pos);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              co[2 * k * d + at[u][0]] = g[u][2 * k] * c.x;
              co[2 * k * d + at[u][1]] = g[u][2 * k + 1] * c.x;
              co[(2 * k + 1) * d + at[u][0]] = -g[u][2 * k + 1] * c.y;
              co[(2 * k + 1) * d + at[u][1]] = g[u][2 * k] * c.y;
            }
          }
      }
      if (lane == 0) {
        StageInfo& f = *reinterpret_cast<StageInfo*>(st);
        f.t = t;
        f.tok = tok;
        f.r0 = r0;
        f.r1 = r1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.full[s]);
    }
    if (*abort)  // copies in flight land (or their time runs out) before the memory goes
      for (int i = n > kTokStages ? n - kTokStages : 0; i < n; ++i)
        mbar_wait_bounded(&bar.full[i % kTokStages], (uint32_t)((i / kTokStages) & 1), 20000000LL);
    return;
  }

  // this lane's entries e0 .. e0 + VE of a row and their partners'
  const int sub = lane % LPR, mine = lane / LPR, e0 = sub * VE, w = e0 - a.rot_start;
  const bool in = half > 0 && w >= 0 && w < a.rot_dim, has = e0 < d;
  const int shift = w < half ? half : -half;
  // whether the norm covers these, their partners (without any, the factor -- NaN perhaps -- meets no partner)
  const bool own = e0 < a.norm_dim, theirs = in && e0 + shift < a.norm_dim;
  int n = 0;
  for (long long it = blockIdx.x; it < items; it += gridDim.x, ++n) {
    const int s = n % kTokStages;
    const bool ok = wait_or_abort(&bar.full[s], (uint32_t)((n / kTokStages) & 1), abort, a.status);
    if (__any_sync(0xffffffffu, !ok)) break;
    const unsigned char* st = stage(s);
    const StageInfo& f = *reinterpret_cast<const StageInfo*>(st);
    if (f.t.live) {
      const int r0 = f.r0, r1 = f.r1;
      const unsigned char* data = st + kInfoBytes + 16 * d;
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {  // queries, keys
        const int lo = k ? nq : 0, end = k ? nq + nk : nq, hi = end < r1 ? end : r1;
        if (hi <= lo || hi <= r0) continue;
        const bool norm = (k ? a.gk : a.gq) != nullptr;
        float A[VE], B[VE];
#pragma unroll
        for (int j = 0; j < VE; j += 4) {
          const float* co = reinterpret_cast<const float*>(st + kInfoBytes) + 2 * k * d + (has ? e0 + j : 0);
          const float4 x = *reinterpret_cast<const float4*>(co), y = *reinterpret_cast<const float4*>(co + d);
          A[j] = x.x, A[j + 1] = x.y, A[j + 2] = x.z, A[j + 3] = x.w;
          B[j] = y.x, B[j + 1] = y.y, B[j + 2] = y.z, B[j + 3] = y.w;
        }
        // the first rows of this kind that the warp takes (it steps through all rows of the item)
        const int skip = (lo - r0 - warp * RPW + W * RPW - RPW) / (W * RPW);
        int rb = r0 + warp * RPW + (lo > r0 && skip > 0 ? skip : 0) * W * RPW;
        const unsigned char* src = data + (rb + mine - r0) * rowb + e0 * ELEM;
        unsigned char* q_to = k ? nullptr : a.q_out + f.tok * a.qos + (size_t)(rb + mine) * rowb;
#pragma unroll 1
        for (; rb < hi; rb += W * RPW) {
          const int r = rb + mine;
          const bool on = has && r >= lo && r < hi;
          uint4 raw = make_uint4(0, 0, 0, 0), other = raw;
          if (on) {
            raw = *reinterpret_cast<const uint4*>(src);
            if (!PAIR) other = *reinterpret_cast<const uint4*>(in ? src + shift * ELEM : bar.zeros);
          }
          float x[VE], y[VE], o[VE];
          Vec<T>::widen(raw, x);
          if (!PAIR) Vec<T>::widen(other, y);
          float inv = 1.f;
          if (norm) {
            float ssq = 0.f;
#pragma unroll
            for (int j = 0; j < VE; ++j) ssq = fmaf(x[j], x[j], ssq);
            if (PART && !own) ssq = 0.f;
#pragma unroll
            for (int off = LPR / 2; off >= 1; off >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, off);
            inv = rsqrtf(fmaf(ssq, a.inv_norm, a.eps));
            if (PART) {
              const float f = own ? inv : 1.f, g = theirs ? inv : 1.f;
#pragma unroll
              for (int j = 0; j < VE; ++j) {
                x[j] *= f;
                if (!PAIR) y[j] *= g;
              }
              inv = 1.f;
            }
          }
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            o[j] = x[j] * A[j];
            if (!PAIR || in) o[j] = fmaf(PAIR ? x[j ^ 1] : y[j], B[j], o[j]);
            o[j] *= inv;
          }
          unsigned char* dst = q_to;
          if (k) dst = on ? row_to<ELEM, NG>(a, f.t, f.tok, r, nq, nk) : nullptr;
          if constexpr (NG > 0) {
            if (k)
              put_row4<VE, LPR, NG>(o, dst, f.t.pos % kCellTokens, sub);
            else if (on && dst != nullptr)
              *reinterpret_cast<uint4*>(dst + e0 * ELEM) = narrow<T>(o);
          } else {
            if (on && dst != nullptr) *reinterpret_cast<uint4*>(dst + e0 * ELEM) = narrow<T>(o);
          }
          src += W * RPW * rowb;
          q_to += W * RPW * rowb;
        }
      }
      if (r1 > nq + nk) {  // values: as they are
        const int v0 = r0 > nq + nk ? r0 : nq + nk;
        const unsigned char* from = data + (r0 < nq + nk ? (nq + nk - r0) * rowb : 0);
        if constexpr (NG > 0) {
          // (every lane takes part in a row's exchange: whole passes, from the first that holds a value row)
          int rb = r0 + warp * RPW;
          if (v0 >= rb + RPW) rb += (v0 - rb + W * RPW - RPW) / (W * RPW) * (W * RPW);
          for (; rb < r1; rb += W * RPW) {
            const int r = rb + mine;
            const bool on = r >= v0 && r < r1;
            float x[VE];
            Vec<T>::widen(on ? *reinterpret_cast<const uint4*>(from + (r - v0) * vrowb + e0 * ELEM) : make_uint4(0, 0, 0, 0), x);
            put_row4<VE, LPR, NG>(x, on ? row_to<ELEM, NG>(a, f.t, f.tok, r, nq, nk) : nullptr, f.t.pos % kCellTokens, sub);
          }
        } else {
          for (int r = r0 + warp * RPW + mine; r < r1; r += W * RPW)
            if (r >= v0 && e0 < a.dv) {
              unsigned char* dst = row_to<ELEM>(a, f.t, f.tok, r, nq, nk);
              if (dst != nullptr)
                *reinterpret_cast<uint4*>(dst + e0 * ELEM) =
                    *reinterpret_cast<const uint4*>(from + (r - v0) * vrowb + e0 * ELEM);
            }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.empty[s]);
  }
}

// Longer rows: a warp a row, NV vectors a lane -- vector i of lane l is vector l + 32 i, the
// next row's loads in flight while this one is turned.  Vectors that neither norm nor
// rotation touch go as they are.  2,048 tokens of 129 latent rows of 576 bf16, 608 MB, take
// 100.4 us, 6.0 TB/s, 0.89 of the copy rate; the warps' own chain of latencies is as long (in
// place, with only the 64 turned entries of a row moved, the same rows took 97).
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kLongWarps) token_long_rows_kernel(const TokenArgs a) {
  constexpr int VE = Vec<T>::N;
  extern __shared__ float2 cs[];  // [rot_dim / 2] cos, sin; then a rotated span a warp
  pdl_release();
  pdl_wait();
  const int tok = blockIdx.x / a.parts, part = blockIdx.x - tok * a.parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Token t = token_of(a, tok, threadIdx.x == 0);
  if (!t.live) return;
  find_pool_rows<sizeof(T)>(a, t);
  const int half = a.rot_dim >> 1;
  for (int i = threadIdx.x; i < half; i += 32 * kLongWarps) cs[i] = turn_cos_sin(t.pos, a.inv_freq[i]);
  __syncthreads();
  float* span = reinterpret_cast<float*>(cs + half) + warp * a.rot_dim;
  const int nq = a.q ? a.Hq : 0, nk = a.k ? a.H : 0, nv = a.v ? a.H : 0;
  const int rows = nq + nk + nv, stride = a.parts * kLongWarps;
  uint4 next[NV];
  const unsigned char* src = nullptr;
  unsigned char *dst = nullptr, *to = nullptr;
  auto load = [&](int r) {  // the next row flies while this one is turned
    if (r >= rows) return;
    src = row_from<sizeof(T)>(a, tok, r, nq, nk);
    dst = row_to<sizeof(T)>(a, t, tok, r, nq, nk);
    const int d = r >= nq + nk ? a.dv : a.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (lane + 32 * i) * VE;
      next[i] = e0 < d ? *reinterpret_cast<const uint4*>(src + (size_t)e0 * sizeof(T)) : make_uint4(0, 0, 0, 0);
    }
  };
  int r = part * kLongWarps + warp;
  load(r);
  for (; r < rows; r += stride) {
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = next[i];
    to = dst;
    load(r + stride);
    const bool is_v = r >= nq + nk;
    const int d = is_v ? a.dv : a.d;
    const unsigned char* gamma = r < nq ? a.gq : is_v ? nullptr : a.gk;
    float inv = 1.f;
    if (gamma != nullptr) {
      float ssq = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((lane + 32 * i) * VE < a.norm_dim) {
          float x[VE];
          Vec<T>::widen(raw[i], x);
#pragma unroll
          for (int j = 0; j < VE; ++j) ssq = fmaf(x[j], x[j], ssq);
        }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, off);
      inv = rsqrtf(fmaf(ssq, a.inv_norm, a.eps));
    }
    const bool turn = half > 0 && !is_v, halves = turn && a.style == SKV_ROPE_HALF;
    if (halves) __syncwarp();  // the row before's partners have been read
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (lane + 32 * i) * VE, w = e0 - a.rot_start;
      const bool in = turn && w >= 0 && w < a.rot_dim, normed = gamma != nullptr && e0 < a.norm_dim;
      if (!in && !normed) continue;
      float x[VE];
      Vec<T>::widen(raw[i], x);
      if (normed) {
        float g[VE];
        Vec<T>::load(gamma + (size_t)e0 * sizeof(T), g);
#pragma unroll
        for (int j = 0; j < VE; ++j) x[j] = x[j] * inv * g[j];
      }
      if (in && halves) {  // finished below, with the partners
#pragma unroll
        for (int j = 0; j < VE; ++j) span[w + j] = x[j];
        continue;
      }
      if (in) {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
          const float2 c = cs[(w + j) >> 1];
          const float u = x[j], z = x[j + 1];
          x[j] = u * c.x - z * c.y;
          x[j + 1] = z * c.x + u * c.y;
        }
      }
      raw[i] = narrow<T>(x);
    }
    if (halves) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int w = (lane + 32 * i) * VE - a.rot_start;
        if (w < 0 || w >= a.rot_dim) continue;
        const bool first = w < half;
        float x[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float2 c = cs[(first ? w : w - half) + j];
          const float o = span[(first ? w + half : w - half) + j];
          x[j] = span[w + j] * c.x + (first ? -o : o) * c.y;
        }
        raw[i] = narrow<T>(x);
      }
    }
    if (to != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e0 = (lane + 32 * i) * VE;
        if (e0 < d) *reinterpret_cast<uint4*>(to + (size_t)e0 * sizeof(T)) = raw[i];
      }
    }
  }
}

// Beside a slot cache: what the append has put into GPU slots goes to the host rows that back
// them as well, else it would be lost when the cache gives the slots to others (it copies
// nothing back).  A warp a (token, KV head), after the append's kernel, so that one is the same
// with and without a cache; at most a row of K and of V a token and head cross the link.  64
// tokens of 8 heads in a graph: 7.1 us in slots, 4.6 without this kernel; 6.3 with every entry
// on the host already, 4.8 without.
__global__ void __launch_bounds__(256) token_backing_kernel(const TokenArgs a, int row_k, int row_v) {
  pdl_release();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5), items = (long long)a.n_tokens * a.H;
  for (long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < items; i += warps) {
    const int tok = (int)(i / a.H), h = (int)(i - (long long)tok * a.H);
    const Token t = token_of(a, tok, false);  // (reported by the append's kernel, bad entries too)
    if (!t.live) continue;
    const int j = t.pos / a.bs, off = t.pos % a.bs, e = table_row(a.pool, t.req, h, a.H)[j];
    if (e < 0 || e >= a.pool.n_gpu) continue;
    // block j of request b: host block b * stride + j of per-head tables, host row b * max_len + t of latent rows
    const long long hb = (long long)t.req * (a.pool.per_head ? a.pool.stride : a.max_len) + j;
    if (hb >= a.pool.n_host) continue;
    const size_t from = gpu_block_row(a.pool, e, h, a.H, a.bs) + off, to = ((size_t)hb * a.H + h) * a.bs + off;
    auto copy = [&](const void* gpu, const void* host, int bytes) {
      const uint4* src = reinterpret_cast<const uint4*>((const unsigned char*)gpu + from * bytes);
      uint4* dst = reinterpret_cast<uint4*>((unsigned char*)const_cast<void*>(host) + to * bytes);
      for (int c = lane; c < bytes / 16; c += 32) dst[c] = src[c];
    };
    copy(a.pool.gpu_k, a.pool.host_k, row_k);
    if (a.v) copy(a.pool.gpu_v, a.pool.host_v, row_v);
  }
}

skv_status launch_backing(const TokenArgs& a, int elem, cudaStream_t st) {
  const long long blocks = ((long long)a.n_tokens * a.H + 7) / 8, most = 8LL * num_sms();
  if (launch_dependent(token_backing_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, st, 1, a,
                       a.d * elem, a.dv * elem) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

int rows_of(const TokenArgs& a) { return (a.q ? a.Hq : 0) + (a.k ? a.H : 0) + (a.v ? a.H : 0); }
// few tokens: as many parts a token as it has rounds of `per` rows, up to about two CTAs an SM
int parts_of(const TokenArgs& a, int per) {
  const long long most = (rows_of(a) + per - 1) / per, want = (2LL * 152 + a.n_tokens - 1) / a.n_tokens;
  return (int)(want < most ? want : most);
}

template <typename T, int LPR, int NG = 0>
skv_status launch_short(TokenArgs& a, cudaStream_t st) {
  const int rows = rows_of(a), wide = (a.v != nullptr && a.dv > a.d ? a.dv : a.d) * (int)sizeof(T);
  const int most = kTokStageMax / wide;  // rows a stage
  a.parts = parts_of(a, kRowWarps<LPR> * (32 / LPR));
  if (a.parts < (rows + most - 1) / most) a.parts = (rows + most - 1) / most;
  a.stage = ((rows + a.parts - 1) / a.parts * wide + 127) & ~127;
  const int smem = kInfoBytes + kTokStages * (kInfoBytes + 16 * a.d + a.stage);
  const bool part = a.norm_dim < a.d && (a.gq != nullptr || a.gk != nullptr);
  const auto kernel = a.style == SKV_ROPE_PAIR
                          ? (part ? token_rows_kernel<T, LPR, true, true, NG> : token_rows_kernel<T, LPR, true, false, NG>)
                          : (part ? token_rows_kernel<T, LPR, false, true, NG> : token_rows_kernel<T, LPR, false, false, NG>);
  const skv_status prep = prepare_kernel((const void*)kernel, kTokSmemMax);
  if (prep != SKV_OK) return prep;
  constexpr int kTurns = 8 * LPR * Vec<T>::N / 2;  // static shared memory
  const int fit = 228 * 1024 / (smem + kTurns + 1024), blocks = fit < kTokCtas<LPR> ? fit : kTokCtas<LPR>;
  const long long items = (long long)a.n_tokens * a.parts, slots = (long long)num_sms() * blocks;
  if (launch_dependent(kernel, dim3((unsigned)(items < slots ? items : slots)), dim3(32 * kRowWarps<LPR> + 32), smem,
                       st, 1, a) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

template <typename T, int NV>
skv_status launch_long(TokenArgs& a, cudaStream_t st) {
  a.parts = parts_of(a, kLongWarps);
  const long long ctas = (long long)a.n_tokens * a.parts;
  if (ctas > 0x7fffffffLL) return SKV_ERR_UNSUPPORTED;
  const size_t smem = (size_t)a.rot_dim * 4 * (1 + kLongWarps);
  if (launch_dependent(token_long_rows_kernel<T, NV>, dim3((unsigned)ctas), dim3(32 * kLongWarps), smem, st, 1, a) !=
      cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

// Staged where a row is a vector a lane, else a warp a row (measured on short rows, too:
// 8,192 tokens of 72 rows of 128 bf16 54 us staged, 289 us a warp a row; 1,237 of 48 rows
// of 128 fp32 13.6 against 17.7).
skv_status launch_rows(TokenArgs& a, bool f32, cudaStream_t st) {
  const int d = a.v != nullptr && a.dv > a.d ? a.dv : a.d;
  if (f32) {
    if (d <= 128) return launch_short<float, 32>(a, st);
    if (d <= 256) return launch_long<float, 2>(a, st);
    if (d <= 640) return launch_long<float, 5>(a, st);
    return launch_long<float, 8>(a, st);
  }
  if (d <= 128) return launch_short<__nv_bfloat16, 16>(a, st);
  if (d <= 256) return launch_short<__nv_bfloat16, 32>(a, st);
  if (d <= 768) return launch_long<__nv_bfloat16, 3>(a, st);
  return launch_long<__nv_bfloat16, 4>(a, st);
}

}  // namespace

skv_status launch_token_rows(const skv_problem& p, const skv_rotary& r, const skv_tokens& t, const PoolView& pool,
                             void* q_out, void* k_out, int32_t* status, cudaStream_t st, bool cached, int group) {
  const int e = p.dtype == SKV_DTYPE_F32 ? 4 : 2;
  TokenArgs a;
  a.q = (const unsigned char*)t.q;
  a.k = (const unsigned char*)t.k;
  a.v = pool.table != nullptr && pool.gpu_v != nullptr ? (const unsigned char*)t.v : nullptr;
  a.qs = t.q_stride * e;
  a.ks = t.k_stride * e;
  a.vs = t.v_stride * e;
  a.q_out = (unsigned char*)q_out;
  a.k_out = (unsigned char*)k_out;
  a.qos = q_out == t.q ? a.qs : (long long)p.n_q_heads * p.d_qk * e;
  a.kos = k_out == t.k ? a.ks : (long long)p.n_kv_heads * p.d_qk * e;
  a.pool = pool;
  a.positions = t.positions;
  a.requests = t.requests;
  a.seq_lens = p.seq_lens;
  a.n_tokens = t.n_tokens;
  a.B = p.batch;
  a.H = p.n_kv_heads;
  a.Hq = p.n_q_heads;
  a.d = p.d_qk;
  a.dv = p.d_v;
  a.max_len = p.max_len;
  a.bs = p.block_size;
  a.rot_start = r.rot_start;
  a.rot_dim = r.rot_dim;
  a.style = r.style;
  a.norm_dim = r.norm_dim > 0 ? r.norm_dim : p.d_qk;
  a.eps = r.eps;
  a.inv_norm = 1.f / (float)a.norm_dim;
  a.inv_freq = r.inv_freq;
  a.gq = (const unsigned char*)r.q_gamma;
  a.gk = (const unsigned char*)r.k_gamma;
  a.status = status;
  a.parts = 1;
  a.stage = 0;
  const bool f32 = p.dtype == SKV_DTYPE_F32;
  if (group > 0) {  // (rows of 128)
    if (f32)
      return group == 32 ? launch_short<float, 32, 4>(a, st)
                         : group == 64 ? launch_short<float, 32, 2>(a, st) : launch_short<float, 32, 1>(a, st);
    return group == 32 ? launch_short<__nv_bfloat16, 16, 4>(a, st)
                       : group == 64 ? launch_short<__nv_bfloat16, 16, 2>(a, st) : launch_short<__nv_bfloat16, 16, 1>(a, st);
  }
  const skv_status rows = launch_rows(a, f32, st);
  return rows == SKV_OK && cached ? launch_backing(a, e, st) : rows;
}

}  // namespace skv
