// k_cache.hip -- the paged key-value cache of the target's side of a round:
// block tables and slots from the requests' lengths, the rows' keys and
// values into their slots, and the accepted path's rows to their places
// behind the context.
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

// ---------------------------------------------------------------------
// Page plan.  With need_b = ceil((ctx_b + n_b + 1) / page), want_b =
// max(need_b - held_b, 0) and back_b = max(held_b - need_b, 0), request b
// takes want_b pages from the free ring at offset sum_{b' < b} want_b' when
// sum_{b' <= b} want_b' is at most the ring's count, and gives back_b pages
// to its tail at offset sum_{b' < b} back_b'.  The free part and the part
// behind it never meet (free and held pages together are at most n_pages),
// so takes and gives of different requests need no order between them.
//
// plan_scan: one workgroup computes both prefix sums and the new state.
// plan_apply: a thread for each row, and the first workgroup of a request
// for its pages.  Both are bound by the latency of a few dependent loads:
// 3.5 and 5 us for 128 requests of 513 rows, whose 1 MB takes 0.2.  Plans of
// few rows and requests run in plan_small, one workgroup that does both (65
// rows of one request 3.2 us instead of 4.2 for the two launches, 16 x 65
// rows 5.2 and 5.8, 64 x 64 rows 9.6 and 6.4; the host's part of a launch is
// 2.5 us more).

constexpr int kScanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kSmallRows = 2048;  // rows of a plan in one workgroup, at most
constexpr int kSmallBatch = 64;   // and requests

__device__ __forceinline__ int64_t pages_for(int64_t tokens, int shift) {
  return (tokens + ((1 << shift) - 1)) >> shift;
}

// x / d and x % d for x >= 0, d > 0; both mostly fit 32 bits, where the
// division is several times shorter.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t d) {
  if (((x | d) >> 32) == 0) return (uint32_t)x / (uint32_t)d;
  return x / d;
}
__device__ __forceinline__ int64_t remainder_of(int64_t x, int64_t d) {
  return x - quotient(x, d) * d;
}

// inclusive prefix sums of two values over the first n threads
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b,
                                            int64_t (*sum)[2], int tid,
                                            int n) {
  const int lane = tid & 63, wave = tid >> 6;
  for (int d = 1; d < kWave && d < n; d <<= 1) {
    const int64_t x = __shfl_up(a, d, kWave), y = __shfl_up(b, d, kWave);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  if (lane == kWave - 1) {
    sum[wave][0] = a;
    sum[wave][1] = b;
  }
  __syncthreads();
  for (int w = 0; w < wave && wave * kWave < n; ++w) {
    a += sum[w][0];
    b += sum[w][1];
  }
}

__device__ __forceinline__ void plan_scan(const PlanArgs& a) {
  __shared__ int64_t sum[kScanThreads / kWave][2];
  __shared__ int64_t total[3];  // wanted, given back, taken
  const int tid = threadIdx.x;
  const PageGeom& g = a.g;
  const int head0 = a.ring_state[0], count0 = a.ring_state[1];
  int head = head0 % g.n_pages;
  head += head < 0 ? g.n_pages : 0;
  const int count = min(max(count0, 0), g.n_pages);
  if (tid == 0) total[0] = total[1] = total[2] = 0;
  for (int b0 = 0; b0 < g.batch; b0 += kScanThreads) {
    __syncthreads();
    const int b = b0 + tid;
    const bool in = b < g.batch;
    int held = 0, n = -1;
    int64_t need = 0;
    if (in) {
      held = min(max(a.held[b], 0), g.max_pages);
      n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
      need = pages_for((int64_t)clamp_ctx(g.ctx_len[b]) + n + 1, g.shift);
    }
    const int to = (int)min(need, (int64_t)g.max_pages);
    const int64_t want = max(to - held, 0), back = max(held - to, 0);
    int64_t wi = want, bi = back;
    block_scan2(wi, bi, sum, tid, min(kScanThreads, g.batch - b0));
    wi += total[0];
    bi += total[1];
    const bool fits = wi <= count;
    __syncthreads();
    if (in) {
      const int after = fits ? to : min(held, to);
      // (offsets into the ring; the first is used only where it fits)
      a.req[b] = make_int4((int)(wi - want),
                           (int)remainder_of(bi - back, g.n_pages), held,
                           after);
      a.held[b] = after;
      a.missing[b] = (int)(need - after);
      if (a.served) a.served[b] = need > after ? -1 : n;
      // the last request that is served has the largest sum
      if (fits && (tid & 63) == 63 - __builtin_clzll(__ballot(fits)))
        atomicMax((unsigned long long*)&total[2], (unsigned long long)wi);
      if (b == g.batch - 1 || tid == kScanThreads - 1) {
        total[0] = wi;
        total[1] = bi;
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.ring0[0] = make_int2(head, count);
    a.ring_state[0] = (int)remainder_of(head + total[2], g.n_pages);
    a.ring_state[1] = (int)min(count - total[2] + total[1],
                               (int64_t)g.n_pages);
  }
}

// Slot and place of row i of request b.
__device__ __forceinline__ void plan_row(const PlanArgs& a, int b, int i) {
  const PageGeom& g = a.g;
  const int4 rq = a.req[b];
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  const int ctx = clamp_ctx(g.ctx_len[b]);
  const int held = rq.z, after = rq.w;
  int64_t s = -1;
  int place = -1;
  if (i <= n) {
    const int p = ctx + i, j = p >> g.shift;
    if (j < after) {
      // pages taken by this call are read where they come from: the table
      // may not hold them yet
      const int page =
          j < held ? a.table[(int64_t)b * g.max_pages + j]
                   : a.ring[remainder_of(
                         (int64_t)a.ring0[0].x + rq.x + j - held, g.n_pages)];
      if (page >= 0 && page < g.n_pages)
        s = ((int64_t)page << g.shift) + (p & ((1 << g.shift) - 1));
    }
    if (a.pos) place = ctx + (i > 0 ? a.depth[(int64_t)b * g.N + i - 1] : 0);
  }
  a.slot[(int64_t)b * (g.N + 1) + i] = s;
  if (a.pos) a.pos[(int64_t)b * (g.N + 1) + i] = place;
}

// Pages that request b takes or gives back, by `threads` threads.
__device__ __forceinline__ void plan_pages(const PlanArgs& a, int b, int t,
                                           int threads) {
  const PageGeom& g = a.g;
  const int4 rq = a.req[b];
  const int2 ring0 = a.ring0[0];
  const int held = rq.z, after = rq.w;
  int32_t* table = a.table + (int64_t)b * g.max_pages;
  for (int j = held + t; j < after; j += threads)
    table[j] =
        a.ring[remainder_of((int64_t)ring0.x + rq.x + j - held, g.n_pages)];
  for (int j = after + t; j < held; j += threads) {
    a.ring[remainder_of((int64_t)ring0.x + ring0.y + rq.y + j - after,
                        g.n_pages)] = table[j];
    table[j] = -1;
  }
}

__global__ __launch_bounds__(kScanThreads) void plan_scan_kernel(PlanArgs a) {
  plan_scan(a);
}

__global__ __launch_bounds__(kApplyThreads) void plan_apply_kernel(
    PlanArgs a) {
  const int b = blockIdx.x, i = blockIdx.y * kApplyThreads + threadIdx.x;
  if (i <= a.g.N) plan_row(a, b, i);
  if (blockIdx.y == 0) plan_pages(a, b, threadIdx.x, kApplyThreads);
}

// all rows over the threads, the requests' pages over the waves
__global__ __launch_bounds__(kScanThreads) void plan_small_kernel(PlanArgs a) {
  plan_scan(a);
  __syncthreads();
  const int tid = threadIdx.x, R = a.g.N + 1;
  for (int x = tid; x < a.g.batch * R; x += kScanThreads)
    plan_row(a, x / R, x % R);
  for (int b = tid >> 6; b < a.g.batch; b += kScanThreads / kWave)
    plan_pages(a, b, tid & 63, kWave);
}

hipError_t launch_cache_plan(const PlanArgs& a, hipStream_t s) {
  if (a.g.batch <= kSmallBatch &&
      (int64_t)a.g.batch * (a.g.N + 1) <= kSmallRows) {
    hipLaunchKernelGGL(plan_small_kernel, dim3(1), dim3(kScanThreads), 0, s,
                       a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(plan_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int pieces = a.g.N / kApplyThreads + 1;
  hipLaunchKernelGGL(plan_apply_kernel, dim3(a.g.batch, pieces),
                     dim3(kApplyThreads), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------
// Row writes: one thread copies a 16-byte piece of a row's key and of its
// value; consecutive threads take consecutive pieces of a row, so a wave's
// loads and stores are whole rows.  Bound by memory: 65,664 rows of 8 heads
// of 128 (538 MB read and written) in 105 us, 5.1 TB/s, what a copy of 1 GiB
// reaches; 64 rows 2.2 us, the latency of the slot, the row and the store.
__global__ __launch_bounds__(256) void cache_write_kernel(WriteArgs a) {
  const int hc = a.D / 8, rc = a.Hkv * hc;  // pieces of a head, of a row
  const int64_t total = a.rows * rc;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = quotient(i, rc);
    const int c = (int)(i - row * rc);
    const int64_t slot = a.slot[row];
    if (slot < 0 || slot >= a.n_slots) continue;
    const int h = c / hc;
    const int64_t page = slot >> a.shift;
    const int64_t off = slot & ((1 << a.shift) - 1);
    const int64_t to =
        (((page * a.Hkv + h) << a.shift) + off) * hc + (c - h * hc);
    a.kc[to] = a.k[row * a.ks + c];
    a.vc[to] = a.v[row * a.vs + c];
  }
}

hipError_t launch_cache_write(const WriteArgs& a, hipStream_t s) {
  const int64_t total = a.rows * a.Hkv * (a.D / 8);
  const int64_t blocks = (total + 255) / 256;
  hipLaunchKernelGGL(cache_write_kernel,
                     dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------
// Commit: node a_j of the accepted path moves to the place of node j.  The
// path is ascending, so a_j >= j: a thread that moves one 16-byte column of
// its request in ascending j, kMove sources loaded before their stores,
// reads every source before anything overwrites it (a later source a_j is
// at least j, past every place written so far), and columns do not touch
// each other.  Moves onto themselves are left out.  A path of the usual
// depth is one round of loads: the time is the latency of the chain lengths
// and nodes -> pages -> rows -> stores, then the bytes (one request of 32
// layers 3.2 us, 32 requests of 16 layers 7.0 us, 32 MB read and written: 4.6
// TB/s).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kMove = 16;
constexpr int kMoveList = 128;  // moves resolved to slots at a time

__global__ __launch_bounds__(256) void cache_commit_kernel(CommitArgs a,
                                                           int write_len) {
  __shared__ int64_t from[kMoveList], to[kMoveList];
  __shared__ int s_end;
  const PageGeom& g = a.g;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int32_t* acc = a.accept + (int64_t)b * a.B;
  const int nd0 = tid < min(kMoveList, a.B) ? acc[tid] : -1;
  const int len = g.ctx_len[b];
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  const int ctx = clamp_ctx(len);
  const int tau = min(max(a.tau[b], 0), a.B + 1);
  if (write_len && blockIdx.x == 0 && tid == 0)
    a.ctx_out[b] = n < 0 ? len : ctx + tau;
  const int moves = n < 0 ? 0 : min(min(tau - 1, a.B), n);
  const int hc = g.D / 8;
  const int cols = a.layers * g.Hkv * hc * 2;
  const int col = blockIdx.x * 256 + tid;
  const bool live = col < cols;
  // column = ((layer * Hkv + head) * 2 + value) * hc + piece
  const int c = live ? col % hc : 0, hkv = live ? col / hc : 0;
  const int lh = hkv >> 1, h = lh % g.Hkv;
  uint4* cache = (hkv & 1) ? a.vc : a.kc;
  cache += (int64_t)(lh / g.Hkv) * a.layer_stride +
           ((int64_t)h << g.shift) * hc + c;
  const int32_t* table = g.table + (int64_t)b * g.max_pages;
  const int64_t page_chunks = ((int64_t)g.Hkv << g.shift) * hc;
  auto place = [&](int64_t p) -> int64_t {  // chunk of a position, -1: none
    const int64_t j = p >> g.shift;
    const int page = j < g.max_pages ? table[j] : -1;
    if (page < 0 || page >= g.n_pages) return -1;
    return page * page_chunks + (p & ((1 << g.shift) - 1)) * hc;
  };
  for (int j0 = 0; j0 < moves; j0 += kMoveList) {
    if (tid == 0) s_end = min(moves - j0, kMoveList);
    __syncthreads();
    const int j = j0 + tid;
    if (tid < kMoveList && j < moves) {
      const int nd = j0 == 0 ? nd0 : acc[j];
      if (nd < 0 || nd >= n) {
        atomicMin(&s_end, tid);
      } else {
        const int64_t f = place((int64_t)ctx + 1 + nd);
        const int64_t t = place((int64_t)ctx + 1 + j);
        from[tid] = nd == j || t < 0 ? -1 : f;
        to[tid] = t;
      }
    }
    __syncthreads();
    const int end = s_end;
    if (live) {
      for (int i0 = 0; i0 < end; i0 += kMove) {
        u32x4 x[kMove];
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
          // (without a move: the first row of the cache, not stored)
          const int64_t f = i0 + u < end ? from[i0 + u] : -1;
          x[u] = *reinterpret_cast<const u32x4*>(cache + (f < 0 ? 0 : f));
        }
#pragma unroll
        for (int u = 0; u < kMove; ++u)
          if (i0 + u < end && from[i0 + u] >= 0)
            *reinterpret_cast<u32x4*>(cache + to[i0 + u]) = x[u];
      }
    }
    if (end < min(moves - j0, kMoveList)) break;
    __syncthreads();
  }
}

// new lengths in place, once every workgroup of the moves has read them
__global__ __launch_bounds__(256) void cache_length_kernel(CommitArgs a) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= a.g.batch) return;
  const int n = a.g.n_nodes ? a.g.n_nodes[b] : a.g.N;
  const int32_t c = a.g.ctx_len[b];
  a.ctx_out[b] = n < 0 ? c : clamp_ctx(c) + min(max(a.tau[b], 0), a.B + 1);
}

hipError_t launch_cache_commit(const CommitArgs& a, hipStream_t s) {
  const bool alias = a.ctx_out == a.g.ctx_len;
  const int64_t cols = (int64_t)a.layers * a.g.Hkv * (a.g.D / 8) * 2;
  hipLaunchKernelGGL(cache_commit_kernel,
                     dim3((unsigned)((cols + 255) / 256), a.g.batch),
                     dim3(256), 0, s, a, alias ? 0 : 1);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !alias) return e;
  hipLaunchKernelGGL(cache_length_kernel, dim3((a.g.batch + 255) / 256),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace pct
