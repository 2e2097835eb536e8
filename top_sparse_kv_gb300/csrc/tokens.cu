// New tokens: per-head RMS norm and rotation of queries and keys in one pass over their
// rows, and the append of K and V rows to the paged pool through the slot table.
//
//   norm      y_j = gamma_j x_j / sqrt(mean_{i < norm_dim} x_i^2 + eps)
//   rotation  (a, b) -> (a cos - b sin, b cos + a sin) at the angle t * inv_freq[i]
//
// Each row is read once and written once.  One CTA holds one token (or a part of its
// rows): the token's cosines and sines are computed once into shared memory and every
// warp then walks rows of the token's heads -- queries, keys, values -- a row spread over
// LPR lanes in 16-byte vectors, so loads and stores are whole 16-byte accesses of
// consecutive lanes and the sum of squares is a butterfly over the row's lanes.
#include "skv_internal.cuh"

namespace skv {
namespace {

constexpr int kTokWarps = 8;
constexpr int kTokThreads = 32 * kTokWarps;

struct TokenArgs {
  const unsigned char *q, *k, *v;
  long long qs, ks, vs;  // bytes from token to token
  unsigned char *q_out, *k_out;
  long long qos, kos;
  PoolView pool;  // append: the pool rows take K and V
  const int32_t *positions, *requests, *seq_lens;
  int n_tokens, B, H, Hq, d, dv, max_len, bs;
  int rot_start, rot_dim, style, norm_dim;
  float eps;
  const float* inv_freq;
  const unsigned char *gq, *gk;
  int32_t* status;
  int parts;  // CTAs a token
};

// cos and sin of t * f: the turn t f / 2 pi as a 64-bit fraction, whose integer product
// with t wraps modulo one turn by itself.  f / 2 pi carries 2^-53 relative error, so the
// turn is off by less than 2^-24 at t = 2^31 and 2^-35 at t = 2^20.  The nearest quarter
// turn comes off in integers too; what is left is at most an eighth of a turn, so its
// fp32 rounding is at most 2^-25 of pi / 4.
__device__ __forceinline__ float2 turn_cos_sin(int t, float f) {
  double u = (double)f * 0.15915494309189533577;  // 1 / (2 pi)
  u -= floor(u);
  const unsigned long long ph = __double2ull_rz(u * 18446744073709551616.0) * (unsigned long long)t;
  const unsigned long long near = ph + (1ull << 61);
  const int quarter = (int)(near >> 62);
  const long long rem = (long long)(near & ((1ull << 62) - 1)) - (1ll << 61);
  float s, c;
  sincospif((float)(int)(rem >> 30) * 1.16415321826934814453e-10f, &s, &c);  // 2^-33: half turns
  const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -cc : cc, quarter >= 2 ? -ss : ss);
}

// LPR lanes a row, NV vectors a lane: vector i of lane `sub` is vector sub + LPR * i.
template <typename T, int LPR, int NV>
__global__ void __launch_bounds__(kTokThreads) token_rows_kernel(const TokenArgs a) {
  constexpr int VE = Vec<T>::N;
  constexpr int RPW = 32 / LPR;  // rows a warp handles at once
  extern __shared__ float2 cs[];  // [rot_dim / 2] cos, sin; then, NV > 1, a rotated span a warp
  pdl_release();
  pdl_wait();
  const int tok = blockIdx.x / a.parts, part = blockIdx.x - tok * a.parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LPR;

  // the token's request and position; padding and out-of-range tokens end here
  const int req = a.requests ? a.requests[tok] : tok;
  if (a.requests && req < 0) return;
  const bool needs_req = a.pool.table != nullptr || a.positions == nullptr || a.requests != nullptr;
  if (needs_req && req >= a.B) {
    if (threadIdx.x == 0) flag(a.status, SKV_DEV_BAD_INDEX);
    return;
  }
  const int pos = a.positions ? a.positions[tok] : a.seq_lens[req] - 1;
  if (pos < 0 || pos >= a.max_len) {
    const bool bad = a.positions ? pos >= 0 : (pos < -1 || pos >= a.max_len);
    if (bad && threadIdx.x == 0) flag(a.status, SKV_DEV_BAD_LENGTH);
    return;
  }
  const int half = a.rot_dim >> 1;
  for (int i = threadIdx.x; i < half; i += kTokThreads) cs[i] = turn_cos_sin(pos, a.inv_freq[i]);
  __syncthreads();
  float* span = reinterpret_cast<float*>(cs + half) + warp * a.rot_dim;

  const int nq = a.q ? a.Hq : 0, nk = a.k ? a.H : 0, nv = a.v ? a.H : 0;
  const int rows = nq + nk + nv;
  for (int r0 = (part * kTokWarps + warp) * RPW; r0 < rows; r0 += a.parts * kTokWarps * RPW) {
    const int r = r0 + lane / LPR;
    const bool is_q = r < nq, is_v = r >= nq + nk;
    const int h = is_q ? r : is_v ? r - nq - nk : r - nq;
    const int d = is_v ? a.dv : a.d;
    const unsigned char* src = nullptr;
    unsigned char* dst = nullptr;
    if (r < rows) {
      src = (is_q ? a.q + tok * a.qs : is_v ? a.v + tok * a.vs : a.k + tok * a.ks) + (size_t)h * d * sizeof(T);
      if (is_q) {
        dst = a.q_out + tok * a.qos + (size_t)h * d * sizeof(T);
      } else if (a.pool.table == nullptr) {
        dst = a.k_out + tok * a.kos + (size_t)h * d * sizeof(T);
      } else {
        const int e = table_row(a.pool, req, h, a.H)[pos / a.bs];
        const int off = pos % a.bs;
        if (e >= 0 && e < a.pool.n_gpu) {
          dst = (unsigned char*)(is_v ? a.pool.gpu_v : a.pool.gpu_k) +
                (gpu_block_row(a.pool, e, h, a.H, a.bs) + off) * d * sizeof(T);
        } else if (e < 0 && a.pool.host_k != nullptr && -(long long)e - 1 < a.pool.n_host) {
          dst = (unsigned char*)(is_v ? a.pool.host_v : a.pool.host_k) +
                (((size_t)(-(long long)e - 1) * a.H + h) * a.bs + off) * d * sizeof(T);
        } else if (sub == 0) {
          flag(a.status, SKV_DEV_BAD_SLOT);
        }
      }
    }
    const unsigned char* gamma = is_q ? a.gq : is_v ? nullptr : a.gk;
    float x[NV][VE];
    float ssq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (sub + LPR * i) * VE;
      if (src != nullptr && e0 < d) {
        Vec<T>::load(src + (size_t)e0 * sizeof(T), x[i]);
        if (e0 < a.norm_dim)
#pragma unroll
          for (int j = 0; j < VE; ++j) ssq = fmaf(x[i][j], x[i][j], ssq);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) x[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) ssq += __shfl_xor_sync(0xffffffffu, ssq, off);
    if (gamma != nullptr) {
      const float inv = 1.f / sqrtf(ssq / (float)a.norm_dim + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e0 = (sub + LPR * i) * VE;
        if (e0 < a.norm_dim) {
          float g[VE];
          Vec<T>::load(gamma + (size_t)e0 * sizeof(T), g);
#pragma unroll
          for (int j = 0; j < VE; ++j) x[i][j] = x[i][j] * inv * g[j];
        }
      }
    }
    // rotation: vector-aligned spans, so a vector is inside or outside as a whole
    if (half > 0 && a.style == SKV_ROPE_PAIR) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int w = (sub + LPR * i) * VE - a.rot_start;
        if (!is_v && w >= 0 && w < a.rot_dim) {
#pragma unroll
          for (int j = 0; j < VE; j += 2) {
            const float2 t = cs[(w + j) >> 1];
            const float u = x[i][j], z = x[i][j + 1];
            x[i][j] = u * t.x - z * t.y;
            x[i][j + 1] = z * t.x + u * t.y;
          }
        }
      }
    } else if (half > 0) {
      if constexpr (NV == 1) {
        const int w = sub * VE - a.rot_start;
        const bool in = w >= 0 && w < a.rot_dim, first = w < half;
        const int from = in ? (first ? lane + half / VE : lane - half / VE) : lane;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float o = __shfl_sync(0xffffffffu, x[0][j], from);
          if (in && !is_v) {
            const float2 t = cs[(first ? w : w - half) + j];
            x[0][j] = x[0][j] * t.x + (first ? -o : o) * t.y;
          }
        }
      } else {
        __syncwarp();  // the previous row's partners have been read
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int w = (sub + LPR * i) * VE - a.rot_start;
          if (w >= 0 && w < a.rot_dim)
#pragma unroll
            for (int j = 0; j < VE; ++j) span[w + j] = x[i][j];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int w = (sub + LPR * i) * VE - a.rot_start;
          if (!is_v && w >= 0 && w < a.rot_dim) {
            const bool first = w < half;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              const float2 t = cs[(first ? w : w - half) + j];
              const float o = span[(first ? w + half : w - half) + j];
              x[i][j] = x[i][j] * t.x + (first ? -o : o) * t.y;
            }
          }
        }
      }
    }
    if (dst != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e0 = (sub + LPR * i) * VE;
        if (e0 < d) {
          __align__(16) T out[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) out[j] = from_float<T>(x[i][j]);  // the one rounding
          *reinterpret_cast<uint4*>(dst + (size_t)e0 * sizeof(T)) = *reinterpret_cast<uint4*>(out);
        }
      }
    }
  }
}

template <typename T, int LPR, int NV>
skv_status launch_rows(TokenArgs& a, cudaStream_t st) {
  const int rows = (a.q ? a.Hq : 0) + (a.k ? a.H : 0) + (a.v ? a.H : 0);
  const int per = kTokWarps * (32 / LPR);  // rows a CTA takes at once
  const int most = (rows + per - 1) / per;
  // few tokens: as many CTAs a token as it has rounds of rows, up to about two CTAs an SM
  long long parts = (2LL * 152 + a.n_tokens - 1) / a.n_tokens;
  a.parts = (int)(parts < most ? parts : most);
  const size_t smem = (size_t)a.rot_dim * 4 + (NV > 1 ? (size_t)kTokWarps * a.rot_dim * 4 : 0);
  const long long ctas = (long long)a.n_tokens * a.parts;
  if (ctas > 0x7fffffffLL) return SKV_ERR_UNSUPPORTED;
  if (launch_dependent(token_rows_kernel<T, LPR, NV>, dim3((unsigned)ctas), dim3(kTokThreads), smem, st, 1, a) !=
      cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

}  // namespace

skv_status launch_token_rows(const skv_problem& p, const skv_rotary& r, const skv_tokens& t, const PoolView& pool,
                             void* q_out, void* k_out, int32_t* status, cudaStream_t st) {
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
  a.inv_freq = r.inv_freq;
  a.gq = (const unsigned char*)r.q_gamma;
  a.gk = (const unsigned char*)r.k_gamma;
  a.status = status;
  a.parts = 1;
  const int d = a.v != nullptr && p.d_v > p.d_qk ? p.d_v : p.d_qk;
  if (p.dtype == SKV_DTYPE_F32) {
    if (d <= 128) return launch_rows<float, 32, 1>(a, st);
    if (d <= 256) return launch_rows<float, 32, 2>(a, st);
    if (d <= 640) return launch_rows<float, 32, 5>(a, st);
    return launch_rows<float, 32, 8>(a, st);
  }
  if (d <= 128) return launch_rows<__nv_bfloat16, 16, 1>(a, st);
  if (d <= 256) return launch_rows<__nv_bfloat16, 32, 1>(a, st);
  if (d <= 768) return launch_rows<__nv_bfloat16, 32, 3>(a, st);
  return launch_rows<__nv_bfloat16, 32, 4>(a, st);
}

}  // namespace skv
