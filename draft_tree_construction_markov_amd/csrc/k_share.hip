// k_share.hip -- which requests of a round share a prefix, found from their
// block tables, and their rows packed by group for shared attention.
//
// A page in the contexts of c requests at place j of their tables stands for
// (j + 1) pages that c - 1 of them need not read again, if what precedes it is
// the same in all: gain_b(j) = (j + 1) (c(table[b][j]) - 1).  Each request
// picks its page of most gain (the first such), so that it joins the requests
// it has the most in common with, whoever else shares less.  Requests of one
// pick whose tables agree up to it are a group.  A table is compared with the
// leader's entry by entry: c only decides what is tried, so tables in which a
// page stands at several places or after other pages cost speed at most.
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

namespace {

constexpr int kShareThreads = 256;   // of a request
constexpr int kPackThreads = 1024;
static_assert(kMaxShareBatch == kPackThreads, "a thread per request");

__device__ __forceinline__ int2 share_lengths(const ShareArgs& a, int b) {
  const PageGeom& g = a.g;
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  return make_int2(clamp_ctx(g.ctx_len[b]), n);
}

// whole pages of request b's context; its root's page is not among them
__device__ __forceinline__ int share_pages(const ShareArgs& a, int b) {
  const PageGeom& g = a.g;
  const int2 len = share_lengths(a, b);
  const int cap = g.max_pages << g.shift;
  return len.y < 0 ? 0 : min(len.x, cap - 1) >> g.shift;
}

// A value that other waves of this workgroup may have written before a
// barrier: read past the L1, as atomics write.
__device__ __forceinline__ int fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void share_count(const ShareArgs& a, int b, int t,
                                            int threads) {
  const int full = share_pages(a, b);
  const int32_t* table = a.g.table + (int64_t)b * a.g.max_pages;
  for (int j = t; j < full; j += threads) {
    const int p = table[j];
    if ((unsigned)p < (unsigned)a.g.n_pages) atomicAdd(&a.count[p], 1);
  }
}

// A wave's part of request b's pick: gains and places in one number, larger
// for more gain, then for an earlier place.  Gains are below 2^41 (2^30
// places, 2^10 requests), of which a place's bits leave 33: past them they
// count as alike.
__device__ __forceinline__ uint64_t share_best(const ShareArgs& a, int b,
                                               int t, int threads) {
  const int full = share_pages(a, b);
  const int32_t* table = a.g.table + (int64_t)b * a.g.max_pages;
  uint64_t best = 0;
  for (int j = t; j < full; j += threads) {
    const int p = table[j];
    if ((unsigned)p >= (unsigned)a.g.n_pages) continue;
    const int c = fresh(a.count + p);
    const uint64_t gain = (uint64_t)(j + 1) * (uint64_t)(c - 1);
    const uint64_t top = gain < (1ull << 33) ? gain : (1ull << 33) - 1;
    const uint64_t key = top << 31 | (uint32_t)(0x7fffffff - j);
    if (gain > 0 && key > best) best = key;
  }
  return best;
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t y = __shfl_xor((unsigned long long)x, d, kWave);
    x = y > x ? y : x;
  }
  return x;
}

// Request b picks: its page and the place there, or none (-1).  One lane.
__device__ __forceinline__ void share_pick(const ShareArgs& a, int b,
                                           uint64_t best) {
  const PageGeom& g = a.g;
  int d = -1;
  if (best != 0 && (int64_t)(best >> 31) << g.shift >= a.least) {
    d = 0x7fffffff - (int)(best & 0x7fffffff);
    atomicMin(&a.lead[g.table[(int64_t)b * g.max_pages + d]], b);
  }
  a.place[b] = d;
  a.size[b] = 0;
}

// Whether thread t's entries of request b agree with its leader's.
__device__ __forceinline__ bool share_agrees(const ShareArgs& a, int b,
                                             int lead, int d, int t,
                                             int threads) {
  const int32_t* x = a.g.table + (int64_t)b * a.g.max_pages;
  const int32_t* y = a.g.table + (int64_t)lead * a.g.max_pages;
  bool same = true;
  for (int j = t; j <= d; j += threads) same = same && x[j] == y[j];
  return same;
}

// Leader of request b by its pick, or -1.
__device__ __forceinline__ int share_lead(const ShareArgs& a, int b) {
  const int d = fresh(a.place + b);
  if (d < 0) return -1;
  const int lead = fresh(a.lead + a.g.table[(int64_t)b * a.g.max_pages + d]);
  return fresh(a.place + lead) == d ? lead : -1;
}

// Results, and the rows packed by group: groups in the order of their
// leaders, requests of a group in theirs.  One workgroup, a thread a request.
__device__ __forceinline__ void share_pack(const ShareArgs& a, int* lead_s,
                                           int* rows_s, int2* at_s,
                                           int2 (*wave_sum)) {
  const PageGeom& g = a.g;
  const int b = threadIdx.x, lane = b & 63, wave = b >> 6;
  const bool in = b < g.batch;
  int2 len = make_int2(0, -1);
  int lead = -1, d = -1;
  if (in) {
    len = share_lengths(a, b);
    lead = fresh(a.joined + b);
    if (lead >= 0 && fresh(a.size + lead) < 2) lead = -1;
    d = lead >= 0 ? fresh(a.place + b) : -1;
    a.leader[b] = lead >= 0 ? lead : b;
    a.shared[b] = (d + 1) << g.shift;
  }
  lead_s[b] = lead;
  rows_s[b] = in && lead >= 0 ? len.y + 1 : 0;
  __syncthreads();
  // rows of the group, and those before this request's
  int before = 0, all = 0;
  for (int x = 0; x < g.batch; ++x) {
    const int r = lead_s[x] == lead && lead >= 0 ? rows_s[x] : 0;
    all += r;
    before += x < b ? r : 0;
  }
  // groups and their rows before this one's, at the leaders
  const bool leads = in && lead == b;
  int2 sum = make_int2(leads ? 1 : 0, leads ? all : 0);
  for (int s = 1; s < kWave; s <<= 1) {
    const int x = __shfl_up(sum.x, s, kWave), y = __shfl_up(sum.y, s, kWave);
    if (lane >= s) sum.x += x, sum.y += y;
  }
  if (lane == kWave - 1) wave_sum[wave] = sum;
  __syncthreads();
  int2 head = make_int2(0, 0);
  for (int w = 0; w < wave; ++w)
    head.x += wave_sum[w].x, head.y += wave_sum[w].y;
  int groups = 0;
  for (int w = 0; w < kPackThreads / kWave; ++w) groups += wave_sum[w].x;
  const int group = head.x + sum.x - 1, first = head.y + sum.y - all;
  if (leads) {
    a.view.groups[group] = make_int4(b, (d + 1) << g.shift, all, first);
    at_s[b] = make_int2(group, first);
  }
  // groups that are not there have no rows
  for (int x = groups + b; x < g.batch; x += kPackThreads)
    a.view.groups[x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (in)
    a.view.req[b] = make_int4(len.x, len.y, d + 1, lead >= 0 ? before : -1);
  if (in) a.view.group_of[b] = lead >= 0 ? at_s[lead] : make_int2(-1, 0);
}

// Rows i = t, t + threads .. of request b into the packed order.
__device__ __forceinline__ void share_rows(const ShareArgs& a, int b, int t,
                                           int threads) {
  const int32_t* at = reinterpret_cast<const int32_t*>(a.view.group_of + b);
  if (fresh(at) < 0) return;
  const int R = a.g.N + 1;
  const int n = share_lengths(a, b).y;
  const int to = fresh(at + 1) + fresh(&a.view.req[b].w);
  for (int i = t; i <= n; i += threads) a.view.rows[to + i] = b * R + i;
}

struct PackLds {
  int lead[kPackThreads], rows[kPackThreads];
  int2 at[kPackThreads], wave_sum[kPackThreads / kWave];
};

__global__ __launch_bounds__(256) void share_clear_kernel(ShareArgs a) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p < a.g.n_pages) {
    a.count[p] = 0;
    a.lead[p] = 0x7fffffff;
  }
}

__global__ __launch_bounds__(kShareThreads) void share_count_kernel(
    ShareArgs a) {
  share_count(a, blockIdx.x, threadIdx.x, kShareThreads);
}

__global__ __launch_bounds__(kShareThreads) void share_pick_kernel(
    ShareArgs a) {
  __shared__ uint64_t best_s[kShareThreads / kWave];
  const int b = blockIdx.x;
  const uint64_t best =
      wave_max64(share_best(a, b, threadIdx.x, kShareThreads));
  if ((threadIdx.x & 63) == 0) best_s[threadIdx.x >> 6] = best;
  __syncthreads();
  if (threadIdx.x != 0) return;
  uint64_t top = 0;
  for (int w = 0; w < kShareThreads / kWave; ++w)
    top = best_s[w] > top ? best_s[w] : top;
  share_pick(a, b, top);
}

__global__ __launch_bounds__(kShareThreads) void share_join_kernel(
    ShareArgs a) {
  const int b = blockIdx.x;
  int lead = share_lead(a, b);
  bool same = true;
  if (lead >= 0)
    same = share_agrees(a, b, lead, a.place[b], threadIdx.x, kShareThreads);
  if (__syncthreads_or(same ? 0 : 1)) lead = -1;
  if (threadIdx.x == 0) {
    a.joined[b] = lead;
    if (lead >= 0) atomicAdd(&a.size[lead], 1);
  }
}

__global__ __launch_bounds__(kPackThreads) void share_pack_kernel(
    ShareArgs a, int with_rows) {
  __shared__ PackLds s;
  share_pack(a, s.lead, s.rows, s.at, s.wave_sum);
  if (!with_rows) return;
  __syncthreads();
  for (int b = threadIdx.x >> 6; b < a.g.batch; b += kPackThreads / kWave)
    share_rows(a, b, threadIdx.x & 63, kWave);
}

__global__ __launch_bounds__(256) void share_rows_kernel(ShareArgs a) {
  share_rows(a, blockIdx.x, blockIdx.y * 256 + threadIdx.x, 256 * gridDim.y);
}

// Small batches and caches: one workgroup does all of it, a wave a request.
__global__ __launch_bounds__(kPackThreads) void share_small_kernel(
    ShareArgs a) {
  __shared__ PackLds s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kWaves = kPackThreads / kWave;
  for (int p = threadIdx.x; p < a.g.n_pages; p += kPackThreads) {
    a.count[p] = 0;
    a.lead[p] = 0x7fffffff;
  }
  __syncthreads();
  for (int b = wave; b < a.g.batch; b += kWaves)
    share_count(a, b, lane, kWave);
  __syncthreads();
  for (int b = wave; b < a.g.batch; b += kWaves) {
    const uint64_t best = wave_max64(share_best(a, b, lane, kWave));
    if (lane == 0) share_pick(a, b, best);
  }
  __syncthreads();
  for (int b = wave; b < a.g.batch; b += kWaves) {
    int lead = share_lead(a, b);
    bool same = true;
    if (lead >= 0)
      same = share_agrees(a, b, lead, fresh(a.place + b), lane, kWave);
    if (__ballot(!same)) lead = -1;
    if (lane == 0) {
      a.joined[b] = lead;
      if (lead >= 0) atomicAdd(&a.size[lead], 1);
    }
  }
  __syncthreads();
  share_pack(a, s.lead, s.rows, s.at, s.wave_sum);
  __syncthreads();
  for (int b = wave; b < a.g.batch; b += kWaves) share_rows(a, b, lane, kWave);
}

constexpr int kSmallTable = 32768;   // table entries,
constexpr int kSmallPages = 16384;   // pages and
constexpr int kPackRows = 16384;     // rows that one workgroup goes through

}  // namespace

hipError_t launch_share(const ShareArgs& a, hipStream_t s) {
  const PageGeom& g = a.g;
  const int64_t rows = (int64_t)g.batch * (g.N + 1);
  if ((int64_t)g.batch * g.max_pages <= kSmallTable &&
      g.n_pages <= kSmallPages && rows <= kPackRows) {
    hipLaunchKernelGGL(share_small_kernel, dim3(1), dim3(kPackThreads), 0, s,
                       a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(share_clear_kernel,
                     dim3((unsigned)(((int64_t)g.n_pages + 255) / 256)),
                     dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 each(g.batch), block(kShareThreads);
  hipLaunchKernelGGL(share_count_kernel, each, block, 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(share_pick_kernel, each, block, 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(share_join_kernel, each, block, 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(share_pack_kernel, dim3(1), dim3(kPackThreads), 0, s, a,
                     rows <= kPackRows ? 1 : 0);
  e = hipGetLastError();
  if (e != hipSuccess || rows <= kPackRows) return e;
  hipLaunchKernelGGL(share_rows_kernel,
                     dim3(g.batch, (unsigned)((g.N + 256) / 256)), dim3(256),
                     0, s, a);
  return hipGetLastError();
}

}  // namespace pct
