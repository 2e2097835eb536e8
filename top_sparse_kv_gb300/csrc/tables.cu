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
};

// Sums of N values over the block's threads before this one; the totals go to all.
template <int N>
__device__ __forceinline__ void block_scan(long long (&a)[N], long long (*warps)[N], long long (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = a[i];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long u = __shfl_up_sync(0xffffffffu, x[i], off);
      if (lane >= off) x[i] += u;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) warps[warp][i] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] -= a[i];
    all[i] = 0;
  }
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (w == warp) x[i] += all[i];
      all[i] += warps[w][i];
    }
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = x[i];
}

__device__ __forceinline__ int saturate(long long x) { return x > 0x7fffffffLL ? 0x7fffffff : (int)x; }

// the last request whose sum is at most i (sums ascend from sums[0] = 0; requests of nothing are passed over)
__device__ __forceinline__ int find(const int* sums, int B, int i) {
  int lo = 0, hi = B;
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
  extern __shared__ int smem[];
  __shared__ long long s_asked[kThreads / 32][3], s_given[kThreads / 32][1];
  __shared__ int s_last;
  const skv_tables& t = a.t;
  const int B = t.batch, bs = t.block_size;
  int* rows = smem;               // [B + 1] rows of the step before each request (saturated)
  int* given = rows + B + 1;      // [B + 1] blocks given to requests before
  int* freed = given + B + 1;     // [B + 1] blocks given back by requests before
  int* start = freed + B + 1;     // [B] first new position; -1: no tokens, or refused
  int* from = start + B;          // [B] table index of its first new block, or of the first it gives back
  int* lens = from + B;           // [B] the new length
  const bool reports = blockIdx.x == 0;
  pdl_release();
  pdl_wait();
  int count = t.state[0];
  count = count < 0 ? 0 : count > t.n_blocks ? t.n_blocks : count;
  const int first = t.base / bs;
  const int per = (B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = b0 + per < B ? b0 + per : B;
  // what each request asks for
  long long asked[3] = {0, 0, 0};  // rows, blocks back, blocks needed
  for (int b = b0; b < b1; ++b) {
    const int L = t.seq_lens[b], n = a.n_new[b];
    const bool bad = L < 0 || L > t.max_len || (L > 0 && L < t.base);
    const int have = !bad && L > t.base ? (int)(((long long)L + bs - 1) / bs) : first;
    lens[b] = L;
    start[b] = -1;
    from[b] = have;
    int need = 0, back = 0;
    if (n != 0 && bad) {
      if (reports) flag(a.status, SKV_DEV_BAD_LENGTH);
    } else if (n > 0) {
      const int s = L == 0 ? t.base : L;
      if (s > t.max_len - n) {
        if (reports) flag(a.status, SKV_DEV_BAD_LENGTH);
      } else {
        start[b] = s;
        need = (int)(((long long)s + n + bs - 1) / bs) - have;
      }
    } else if (n < 0) {
      const long long left = (long long)L + n;
      const int keep = left > t.base ? (int)((left + bs - 1) / bs) : first;
      lens[b] = left > t.base ? (int)left : 0;
      from[b] = keep;
      back = have - keep;
    }
    given[b] = need;
    freed[b] = back;
    asked[0] += n > 0 ? n : 0;
    asked[1] += back;
    asked[2] += need;
  }
  long long all[3], all_given[1];
  block_scan<3>(asked, s_asked, all);
  // who gets it
  long long before[1] = {0};
  const long long free = count + all[1];
  for (int b = b0; b < b1; ++b) {
    const int n = a.n_new[b], need = given[b], back = freed[b];
    asked[2] += need;
    rows[b] = saturate(asked[0]);
    freed[b] = saturate(asked[1]);
    asked[0] += n > 0 ? n : 0;
    asked[1] += back;
    if (start[b] >= 0) {
      const bool fits = asked[0] <= a.n_tokens, blocks = need == 0 || asked[2] <= free;
      if (!fits && reports) flag(a.status, SKV_DEV_BAD_INDEX);
      if (fits && !blocks && reports) flag(a.status, SKV_DEV_NO_BLOCK);
      if (fits && blocks) {
        lens[b] = start[b] + n;
      } else {
        start[b] = -1;
        given[b] = 0;
      }
    }
    before[0] += given[b];
  }
  block_scan<1>(before, s_given, all_given);
  for (int b = b0; b < b1; ++b) {
    const int g = given[b];
    given[b] = saturate(before[0]);
    before[0] += g;
  }
  if (threadIdx.x == 0) {
    rows[B] = saturate(all[0]);
    given[B] = saturate(all_given[0]);
    freed[B] = saturate(all[1]);
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
  // the slot map: four rows a thread, one bisection
  for (long long r0 = me * 4; r0 < a.n_tokens; r0 += step * 4) {
    int pos[4], req[4];
    long long slot[4];
    int b = r0 < rows[B] ? find(rows, B, (int)r0) : B;
    int last = -1, e = 0;  // the table index that e was found for (of request b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long r = r0 + i;
      pos[i] = req[i] = -1;
      slot[i] = -1;
      if (r >= a.n_tokens || r >= rows[B]) continue;
      while (b + 1 < B && rows[b + 1] <= r) ++b, last = -1;
      if (start[b] < 0) continue;
      const int p = start[b] + (int)(r - rows[b]);
      pos[i] = p;
      req[i] = b;
      if (a.slots != nullptr) {
        const int j = p / bs;
        if (j != last) {
          e = j < from[b] ? t.slot_table[(size_t)b * t.table_stride + j] : block_at(given[b] + j - from[b]);
          last = j;
        }
        slot[i] = (long long)e * bs + (p - j * bs);
      }
    }
    if (r0 + 4 <= a.n_tokens) {
      *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.requests + r0) = make_int4(req[0], req[1], req[2], req[3]);
      if (a.slots != nullptr) {
        *reinterpret_cast<longlong2*>(a.slots + r0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(a.slots + r0 + 2) = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < a.n_tokens) {
          a.positions[r0 + i] = pos[i];
          a.requests[r0 + i] = req[i];
          if (a.slots != nullptr) a.slots[r0 + i] = slot[i];
        }
    }
  }
  // new table entries
  for (long long i = me; i < K; i += step) {
    const int b = find(given, B, (int)i);
    t.slot_table[(size_t)b * t.table_stride + from[b] + ((int)i - given[b])] = block_at((int)i);
  }
  // the stack takes what is left of the blocks given back
  for (long long i = me; i < (long long)R - K; i += step) {
    const int e = back_at(R - 1 - (int)i);
    if (count + i < t.n_blocks)
      t.free_blocks[count + i] = e;
    else
      flag(a.status, SKV_DEV_BAD_SLOT);
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
  TableArgs a{t, n_new, n_tokens, positions, requests, reinterpret_cast<long long*>(slots), status};
  const int smem = 6 * 4 * (t.batch + 1);
  const skv_status prep = prepare_kernel((const void*)update_tables_kernel, 6 * 4 * (kMaxBatch + 1));
  if (prep != SKV_OK) return prep;
  // A sweep of rows a CTA, or of the blocks that come with them, two CTAs a SM at most.  Without rows
  // the call gives blocks back, how many is known on the device only: as for all that the tables
  // hold, a CTA a SM at most.
  const long long entries = (long long)t.batch * t.table_stride;
  const long long blocks = n_tokens > 0 ? n_tokens / t.block_size + t.batch : entries < t.n_blocks ? entries : t.n_blocks;
  long long ctas = ((long long)n_tokens + 4 * kThreads - 1) / (4 * kThreads), more = (blocks + 8 * kThreads - 1) / (8 * kThreads);
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
