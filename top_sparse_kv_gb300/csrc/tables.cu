// Block tables and slot maps from request lengths: one kernel a step.
//
// Per request, with its old length L and n new tokens: the rows of its tokens, the blocks it
// needs (or gives back) and whether it can have them all follow from sums over the requests
// before it.  Every CTA makes those sums for itself (a batch is a few thousand words at most,
// read from L2), keeps them in shared memory and takes its share of the outputs: rows of the
// slot map, new table entries, blocks going back onto the stack; each finds its request by
// bisection.  A new block is computed where it is needed rather than read back from the
// table, so no CTA waits for another's writes; lengths and the stack's count, which all of them
// read, are written when all of them have: by the first CTA of a cluster after its barrier, of
// more CTAs by the last to finish (a ticket in the state).
//
// A call is a chain of latencies: 64 requests' step 5 us (its lengths, two sums, its blocks, the
// stores), 8 with nothing in the caches.  256 requests' prompts to 8,192 tokens, 1.1 million rows
// of 16 bytes, take 18 us on 304 CTAs (152: 19, 76: 27), their blocks' way back 8: every CTA's own
// sums, 600 instructions a warp, are two fifths of the first's, a bisection a four rows most of
// the rest.
#include "skv_internal.cuh"

namespace skv {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBatch = 4096;
constexpr unsigned kCluster = 8;  // as many CTAs are one cluster, and wait for each other by its barrier

struct TableArgs {
  skv_tables t;
  const int32_t* n_new;
  int n_tokens;
  int32_t *positions, *requests;
  long long* slots;
  int32_t* status;
  int shift;  // log2 of the tokens of a block, or -1
};

// A short call is over before all its instructions have been fetched (64 requests and their 64
// tokens: 7 us with the loops below unrolled and sums in 64 bits, most of it fetching), so there is
// one copy of everything.  Sums are held at 2^31 - 1: what lies past it is past every limit.
__device__ __forceinline__ unsigned add(unsigned x, unsigned y) { return min(x + y, 0x7fffffffu); }

// Sums of N values over the block's threads before this one; the totals go to all.
template <int N>
__device__ __forceinline__ void block_scan(unsigned (&a)[N], unsigned (*warps)[kThreads / 32], unsigned (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = a[i];
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const unsigned u = __shfl_up_sync(0xffffffffu, x[i], off);
        if (lane >= off) x[i] = add(x[i], u);
      }
    if (level == 1) break;
    if (lane == 31)
#pragma unroll
      for (int i = 0; i < N; ++i) warps[i][warp] = x[i];
    __syncthreads();
    // this thread's own, to be kept; then the warps' sums
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned own = __shfl_up_sync(0xffffffffu, x[i], 1);
      a[i] = lane ? own : 0u;
      x[i] = lane < kThreads / 32 ? warps[i][lane] : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const unsigned before = __shfl_sync(0xffffffffu, x[i], warp ? warp - 1 : 0);
    if (warp) a[i] = add(a[i], before);
    all[i] = __shfl_sync(0xffffffffu, x[i], kThreads / 32 - 1);
  }
}

// the last request whose sum is at most i (sums ascend from sums[0] = 0; requests of nothing are passed over)
__device__ __forceinline__ int find(const unsigned* sums, int B, unsigned i) {
  int lo = 0, hi = B;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 2) update_tables_kernel(const TableArgs a) {
  extern __shared__ unsigned smem[];
  __shared__ unsigned s_asked[3][kThreads / 32], s_given[1][kThreads / 32];
  __shared__ int s_last;
  const skv_tables& t = a.t;
  const int B = t.batch, bs = t.block_size;
  unsigned* rows = smem;              // [B + 1] rows of the step before each request
  unsigned* given = rows + B + 1;     // [B + 1] blocks given to requests before
  unsigned* freed = given + B + 1;    // [B + 1] blocks given back by requests before
  int* start = reinterpret_cast<int*>(freed + B + 1);  // [B] first new position; -1: no tokens, or refused
  int* from = start + B;              // [B] table index of its first new block, or of the first it gives back
  int* lens = from + B;               // [B] the new length
  const bool reports = blockIdx.x == 0;
  auto blocks_of = [&](int n) {  // that hold n tokens
    return a.shift >= 0 ? (int)(((unsigned)n + (unsigned)bs - 1) >> a.shift) : (int)(((unsigned)n + (unsigned)bs - 1) / (unsigned)bs);
  };
  pdl_release();
  pdl_wait();
  int count = t.state[0];
  count = count < 0 ? 0 : count > t.n_blocks ? t.n_blocks : count;
  const int first = t.base / bs;
  const int per = (B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = b0 + per < B ? b0 + per : B;
  // what each request asks for
  unsigned asked[3] = {0, 0, 0};  // rows, blocks back, blocks needed
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int L = t.seq_lens[b], n = a.n_new[b];
    const bool bad = L < 0 || L > t.max_len || (L > 0 && L < t.base);
    const int have = !bad && L > t.base ? blocks_of(L) : first;
    int need = 0, back = 0, s = -1, at = have, len = L;
    if (n != 0 && bad) {
      if (reports) flag(a.status, SKV_DEV_BAD_LENGTH);
    } else if (n > 0) {
      s = L == 0 ? t.base : L;
      if (s > t.max_len - n) {
        s = -1;
        if (reports) flag(a.status, SKV_DEV_BAD_LENGTH);
      } else {
        need = blocks_of(s + n) - have;
      }
    } else if (n < 0) {
      const long long left = (long long)L + n;
      len = left > t.base ? (int)left : 0;
      at = len > 0 ? blocks_of(len) : first;
      back = have - at;
    }
    lens[b] = len;
    start[b] = s;
    from[b] = at;
    given[b] = need;
    freed[b] = back;
    asked[0] = add(asked[0], n > 0 ? n : 0);
    asked[1] = add(asked[1], back);
    asked[2] = add(asked[2], need);
  }
  unsigned all[3], all_given[1], before[1] = {0};
  block_scan<3>(asked, s_asked, all);
  // who gets it
  const unsigned free = add((unsigned)count, all[1]);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int n = a.n_new[b], need = given[b], back = freed[b];
    rows[b] = asked[0];
    freed[b] = asked[1];
    asked[0] = add(asked[0], n > 0 ? n : 0);
    asked[1] = add(asked[1], back);
    asked[2] = add(asked[2], need);
    if (start[b] >= 0) {
      const bool fits = asked[0] <= (unsigned)a.n_tokens, blocks = need == 0 || asked[2] <= free;
      if (!(fits && blocks) && reports) flag(a.status, fits ? SKV_DEV_NO_BLOCK : SKV_DEV_BAD_INDEX);
      if (fits && blocks) {
        lens[b] = start[b] + n;
      } else {
        start[b] = -1;
        given[b] = 0;
      }
    }
    before[0] = add(before[0], given[b]);
  }
  block_scan<1>(before, s_given, all_given);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const unsigned g = given[b];
    given[b] = before[0];
    before[0] = add(before[0], g);
  }
  if (threadIdx.x == 0) {
    rows[B] = all[0];
    given[B] = all_given[0];
    freed[B] = all[1];
  }
  __syncthreads();
  const int K = given[B], R = freed[B];

  // the i-th block given back, the first request's lowest first
  auto back_at = [&](int i) {
    const int b = find(freed, B, i);
    const int e = t.slot_table[(size_t)b * t.table_stride + from[b] + (i - freed[b])];
    if (e < 0 || e >= t.n_blocks) flag(a.status, SKV_DEV_BAD_SLOT);
    return e;
  };
  // the i-th block given out
  auto block_at = [&](int i) { return i < R ? back_at(i) : t.free_blocks[count - 1 - (i - R)]; };

  const long long step = (long long)gridDim.x * kThreads, me = (long long)blockIdx.x * kThreads + threadIdx.x;
  // the slot map: a row a thread, or four where there are more rows than threads: then of one or two
  // requests mostly, and of two blocks at most where a block is four tokens or more
  const int width = a.n_tokens > step ? 4 : 1;
#pragma unroll 1
  for (long long r0 = me * width; r0 < a.n_tokens; r0 += step * width) {
    const int last = (int)(a.n_tokens - r0 < width ? a.n_tokens - r0 : width);
#pragma unroll 1
    for (int i = 0; i < last;) {  // runs of one request's rows, or of none
      const int b = r0 + i < rows[B] ? find(rows, B, (unsigned)(r0 + i)) : B;
      const int end = b < B && rows[b + 1] < r0 + last ? (int)(rows[b + 1] - r0) : last, n = end - i;
      const bool on = b < B && start[b] >= 0;
      int p = on ? start[b] + (int)(r0 + i - rows[b]) : 0;
      // the blocks of the run's first and last row
      int e[2] = {0, 0}, j0 = 0;
      if (on && a.slots != nullptr) {
        j0 = a.shift >= 0 ? p >> a.shift : p / bs;
        const int j1 = blocks_of(p + n) - 1;
#pragma unroll 1
        for (int j = j0; j <= j1; j += j1 > j0 ? j1 - j0 : 1) {
          const int x = j < from[b] ? t.slot_table[(size_t)b * t.table_stride + j] : block_at(given[b] + j - from[b]);
          if (j == j0) e[0] = x;
          e[1] = x;
        }
      }
      if (n == 4 && bs >= 4) {
        const long long r = r0;
        *reinterpret_cast<int4*>(a.positions + r) = on ? make_int4(p, p + 1, p + 2, p + 3) : make_int4(-1, -1, -1, -1);
        const int q = on ? b : -1;
        *reinterpret_cast<int4*>(a.requests + r) = make_int4(q, q, q, q);
        if (a.slots != nullptr) {
          long long s[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int in = p + k - j0 * bs;
            s[k] = !on ? -1 : in < bs ? (long long)e[0] * bs + in : (long long)e[1] * bs + (in - bs);
          }
          *reinterpret_cast<longlong2*>(a.slots + r) = make_longlong2(s[0], s[1]);
          *reinterpret_cast<longlong2*>(a.slots + r + 2) = make_longlong2(s[2], s[3]);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < n; ++k, ++p) {
          const long long r = r0 + i + k;
          a.positions[r] = on ? p : -1;
          a.requests[r] = on ? b : -1;
          if (a.slots != nullptr) {
            int in = p - j0 * bs, x = in < bs ? e[0] : e[1];
            if (on && bs < 4) {  // more than two blocks in a run
              const int j = p / bs;
              x = j < from[b] ? t.slot_table[(size_t)b * t.table_stride + j] : block_at(given[b] + j - from[b]);
              in = p - j * bs;
            }
            a.slots[r] = on ? (long long)x * bs + (in < bs ? in : in - bs) : -1;
          }
        }
      }
      i = end;
    }
  }
  // new table entries; then the stack takes what is left of the blocks given back
#pragma unroll 1
  for (long long i = me; i < K || i < (long long)R - K; i += step) {
    const bool out = i < K;
    const int e = block_at(out ? (int)i : R - 1 - (int)i);
    if (out) {
      const int b = find(given, B, (int)i);
      t.slot_table[(size_t)b * t.table_stride + from[b] + ((int)i - given[b])] = e;
    }
    if (i < (long long)R - K) {
      const int f = out ? back_at(R - 1 - (int)i) : e;
      if (count + i < t.n_blocks)
        t.free_blocks[count + i] = f;
      else
        flag(a.status, SKV_DEV_BAD_SLOT);
    }
  }
  // lengths and the count, once every CTA has read them
  __syncthreads();
  if (gridDim.x > kCluster) {
    if (threadIdx.x == 0) {
      __threadfence();
      s_last = atomicAdd(&t.state[1], 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
  } else if (gridDim.x > 1) {
    cluster_sync();
    if (blockIdx.x > 0) return;
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) t.seq_lens[b] = lens[b];
  if (threadIdx.x == 0) {
    const long long left = (long long)count + R - K;
    t.state[0] = left < t.n_blocks ? (int)left : t.n_blocks;
    if (gridDim.x > kCluster) t.state[1] = 0;
  }
}

}  // namespace

int tables_max_batch() { return kMaxBatch; }

skv_status launch_update_tables(const skv_tables& t, const int32_t* n_new, int n_tokens, int32_t* positions,
                                int32_t* requests, int64_t* slots, int32_t* status, cudaStream_t st) {
  TableArgs a{t, n_new, n_tokens, positions, requests, reinterpret_cast<long long*>(slots), status, -1};
  for (int i = 0; i < 31; ++i)
    if (t.block_size == 1 << i) a.shift = i;
  const int smem = 6 * 4 * (t.batch + 1);
  const skv_status prep = prepare_kernel((const void*)update_tables_kernel, 6 * 4 * (kMaxBatch + 1));
  if (prep != SKV_OK) return prep;
  // A sweep of rows a CTA, two CTAs a SM at most; the new blocks that come with them are fewer.  Without rows
  // the call gives blocks back, how many is known on the device only: a sweep of a sixteenth of what
  // the tables hold, a CTA a SM at most.  Blocks given back in a call that has rows too are not counted: 64
  // rows are one CTA's, which also takes back what a request leaves that goes in the same step (131,072
  // tokens in blocks of 16: 19 us, the step alone 6; a million tokens: 110).
  const long long entries = (long long)t.batch * t.table_stride;
  const long long blocks = n_tokens > 0 ? 0 : entries < t.n_blocks ? entries : t.n_blocks;
  long long ctas = ((long long)n_tokens + 4 * kThreads - 1) / (4 * kThreads), more = (blocks + 16 * kThreads - 1) / (16 * kThreads);
  if (more > num_sms()) more = num_sms();
  if (ctas < more) ctas = more;
  if (ctas < 1) ctas = 1;
  if (ctas > 2 * num_sms()) ctas = 2 * num_sms();
  if (launch_dependent(update_tables_kernel, dim3((unsigned)ctas), dim3(kThreads), (size_t)smem, st,
                       ctas <= kCluster ? (int)ctas : 1, a) != cudaSuccess)
    return SKV_ERR_CUDA;
  SKV_LAUNCH_CHECK();
  return SKV_OK;
}

}  // namespace skv
