// k_share.hip -- which requests of a round share a prefix, found from their
// block tables, and their rows packed by group for shared attention.
//
// A page that c requests have at place j of their tables, all within their
// contexts, stands for (j + 1) pages that c - 1 of them need not read again,
// if what precedes it is the same in all: gain = (j + 1) (c - 1).  Each
// request picks its place of most gain (the first such), so that it joins the
// requests it has the most in common with, whoever else shares less.  Requests
// of one page and place are a group as far as their tables agree up to it,
// entry by entry, with the first one's: c only decides what is tried.
//
// columns: workgroups of 4 places hold the tables' columns in LDS and
// count by comparison (pages counted by atomics took 12 us for 128 tables of
// up to 1281 pages, at 40 holders a page); pick: the best of all columns;
// join: leaders, and the comparison with them; pack: one workgroup.  Each is
// a few dependent loads (128 tables of up to 1281 pages: 6.4, 4.0, 4.4 and 5.6
// us); small tables go through all of it in one workgroup (8 tables of up to 82
// pages 6.9 us).
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

namespace {

constexpr int kShareThreads = 256;   // of a request, of columns
constexpr int kPackThreads = 1024;
constexpr int kWide = 2;             // log2 of the places of columns
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
// barrier: read past the L1.
__device__ __forceinline__ int fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Gain and place in one number, larger for more gain, then for an earlier
// place.  Gains are below 2^41 (2^30 places, 2^10 requests), of which a
// place's bits leave 33: past them they count as alike.
__device__ __forceinline__ uint64_t pick_key(int j, int c) {
  const uint64_t gain = (uint64_t)(j + 1) * (uint64_t)(c - 1);
  const uint64_t top = gain < (1ull << 33) ? gain : (1ull << 33) - 1;
  return top == 0 ? 0 : top << 31 | (uint32_t)(0x7fffffff - j);
}

// Places j0 .. j0 + 2^wide - 1 of all tables, by the whole workgroup (of a
// multiple of so many threads): entries to col [batch][2^wide] (-1: none),
// then the best key of each request to best_s.  full_s: whole pages of the
// requests.  A thread's entries are all at one place, so that a column's
// entry is read once for kMine comparisons.
template <int kMine>
__device__ __forceinline__ void share_columns(const ShareArgs& a, int j0,
                                              int wide, const int* full_s,
                                              int* col,
                                              unsigned long long* best_s) {
  const PageGeom& g = a.g;
  const int w = threadIdx.x & ((1 << wide) - 1), j = j0 + w;
  const int first = threadIdx.x >> wide, step = blockDim.x >> wide;
  const int at = min(j, g.max_pages - 1);
  __syncthreads();
  for (int b0 = first; b0 < g.batch; b0 += kMine * step) {
    int p[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k)
      p[k] = g.table[(int64_t)min(b0 + k * step, g.batch - 1) * g.max_pages +
                     at];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int b = b0 + k * step;
      if (b < g.batch)
        col[b << wide | w] =
            j < full_s[b] && (unsigned)p[k] < (unsigned)g.n_pages ? p[k] : -1;
    }
  }
  __syncthreads();
  for (int b0 = first; b0 < g.batch; b0 += kMine * step) {
    int mine[kMine], count[kMine];
    bool any = false;
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int b = b0 + k * step;
      mine[k] = b < g.batch ? col[b << wide | w] : -1;
      any = any || mine[k] >= 0;
      count[k] = 0;
    }
    if (!any) continue;
#pragma unroll 8
    for (int x = 0; x < g.batch; ++x) {
      const int p = col[x << wide | w];
#pragma unroll
      for (int k = 0; k < kMine; ++k) count[k] += p == mine[k] ? 1 : 0;
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const uint64_t key = mine[k] < 0 ? 0 : pick_key(j, count[k]);
      if (key != 0) atomicMax(&best_s[b0 + k * step], key);
    }
  }
}

// Request b's place by its best key, or none (-1).
__device__ __forceinline__ int share_place(const ShareArgs& a, uint64_t best) {
  return best != 0 && (int64_t)(best >> 31) << a.g.shift >= a.least
             ? 0x7fffffff - (int)(best & 0x7fffffff)
             : -1;
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

// Lowest of thread t's requests that picked the page of request b, place d.
__device__ __forceinline__ int share_lead(const ShareArgs& a, int b, int d,
                                          const int* place, int t,
                                          int threads) {
  const int32_t* at = a.g.table + d;
  const int page = at[(int64_t)b * a.g.max_pages];
  int lead = b;
  for (int x = t; x < b; x += threads)
    if (place[x] == d && at[(int64_t)x * a.g.max_pages] == page)
      lead = min(lead, x);
  return lead;
}

// Results, and the rows packed by group: groups in the order of their
// leaders, requests of a group in theirs.  One workgroup, a thread a request.
struct PackLds {
  int2 lead[kPackThreads];  // leader or -1, rows in a group
  int to[kPackThreads], size[kPackThreads];
  int2 group[kPackThreads], wave_sum[kPackThreads / kWave];
  float totals[kPackThreads / kWave][3];
};
__device__ __forceinline__ void share_pack(const ShareArgs& a, PackLds& s,
                                           bool with_rows) {
  const PageGeom& g = a.g;
  const int b = threadIdx.x, lane = b & 63, wave = b >> 6;
  const bool in = b < g.batch;
  int2 len = make_int2(0, -1);
  int lead = -1, d = -1;
  s.size[b] = 0;
  if (in) {
    len = share_lengths(a, b);
    lead = fresh(a.joined + b);
    d = fresh(a.place + b);
  }
  __syncthreads();
  if (lead >= 0) atomicAdd(&s.size[lead], 1);
  __syncthreads();
  if (lead >= 0 && s.size[lead] < 2) lead = -1;
  if (lead < 0) d = -1;
  s.lead[b] = make_int2(lead, lead >= 0 ? len.y + 1 : 0);
  __syncthreads();
  // rows of the group, and those before this request's
  int before = 0, all = 0;
  if (lead >= 0) {
#pragma unroll 8
    for (int x = 0; x < g.batch; ++x) {
      const int2 y = s.lead[x];
      const int r = y.x == lead ? y.y : 0;
      all += r;
      before += x < b ? r : 0;
    }
  }
  // groups and their rows before this one's, at the leaders
  const bool leads = in && lead == b;
  int2 sum = make_int2(leads ? 1 : 0, leads ? all : 0);
  for (int k = 1; k < kWave; k <<= 1) {
    const int x = __shfl_up(sum.x, k, kWave), y = __shfl_up(sum.y, k, kWave);
    if (lane >= k) sum.x += x, sum.y += y;
  }
  if (lane == kWave - 1) s.wave_sum[wave] = sum;
  __syncthreads();
  int2 head = make_int2(0, 0);
  int groups = 0;
  for (int w = 0; w < kPackThreads / kWave; ++w) {
    const int2 x = s.wave_sum[w];
    groups += x.x;
    if (w < wave) head.x += x.x, head.y += x.y;
  }
  if (leads) {
    const int2 group = make_int2(head.x + sum.x - 1, head.y + sum.y - all);
    a.view.groups[group.x] = make_int4(b, (d + 1) << g.shift, all, group.y);
    s.group[b] = group;
  }
  // groups that are not there have no rows
  if (groups + b < g.batch) a.view.groups[groups + b] = make_int4(0, 0, 0, 0);
  __syncthreads();
  if (in) {
    const int2 group = lead >= 0 ? s.group[lead] : make_int2(-1, 0);
    a.leader[b] = lead >= 0 ? lead : b;
    a.shared[b] = (d + 1) << g.shift;
    a.view.req[b] = make_int4(len.x, len.y, d + 1, lead >= 0 ? before : -1);
    a.view.group_of[b] = group;
    s.to[b] = group.y + before;
  }
  // (only how the attention divides its workgroups depends on these)
  float own = 0.f, rows = 0.f;
  if (len.y >= 0) {
    const int cap = g.max_pages << g.shift, before_own = (d + 1) << g.shift;
    own = (float)(min(min(len.x, cap - 1) + len.y + 1, cap) - before_own);
    rows = (float)(len.y + 1) * (float)before_own;
  }
  if (wave * kWave < g.batch) {
    own = wave_sum(own);
    rows = wave_sum(rows);
    const float requests = (float)__popcll(__ballot(len.y >= 0));
    if (lane == 0) {
      s.totals[wave][0] = own;
      s.totals[wave][1] = requests;
      s.totals[wave][2] = rows;
    }
  }
  __syncthreads();
  if (b < 3) {
    float sum = 0.f;
    for (int w = 0; w * kWave < g.batch; ++w) sum += s.totals[w][b];
    a.view.totals[b] = sum;
  }
  if (!with_rows) return;
  const int R = g.N + 1;
  for (int x = b; x < g.batch * R; x += kPackThreads) {
    const int q = x / R, i = x - q * R;
    if (i < s.lead[q].y) a.view.rows[s.to[q] + i] = x;
  }
}

template <int kMine>
__global__ __launch_bounds__(kShareThreads) void share_columns_kernel(
    ShareArgs a) {
  extern __shared__ unsigned long long dyn[];
  unsigned long long* best_s = dyn;
  int* full_s = reinterpret_cast<int*>(best_s + a.g.batch);
  int* col = full_s + a.g.batch;
  __shared__ int most;
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  int here = 0;
  for (int b = threadIdx.x; b < a.g.batch; b += kShareThreads) {
    const int full = share_pages(a, b);
    best_s[b] = 0;
    full_s[b] = full;
    here = max(here, full);
  }
  here = wave_max(here);
  if ((threadIdx.x & 63) == 0) atomicMax(&most, here);
  __syncthreads();
  const int end = most;
  for (int j0 = blockIdx.x << kWide; j0 < end; j0 += gridDim.x << kWide)
    share_columns<kMine>(a, j0, kWide, full_s, col, best_s);
  __syncthreads();
  for (int b = threadIdx.x; b < a.g.batch; b += kShareThreads)
    a.best[(int64_t)blockIdx.x * a.g.batch + b] = best_s[b];
}

__global__ __launch_bounds__(kWave) void share_pick_kernel(ShareArgs a,
                                                           int columns) {
  const int b = blockIdx.x;
  unsigned long long best = 0;
  for (int w = threadIdx.x; w < columns; w += kWave)
    best = max(best, (unsigned long long)a.best[(int64_t)w * a.g.batch + b]);
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) best = max(best, __shfl_xor(best, k, kWave));
  if (threadIdx.x == 0) a.place[b] = share_place(a, best);
}

__global__ __launch_bounds__(kShareThreads) void share_join_kernel(
    ShareArgs a) {
  __shared__ int lead_s;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int d = a.place[b];
  if (d < 0) {
    if (tid == 0) a.joined[b] = -1;
    return;
  }
  if (tid == 0) lead_s = b;
  __syncthreads();
  const int mine = share_lead(a, b, d, a.place, tid, kShareThreads);
  if (mine < b) atomicMin(&lead_s, mine);
  __syncthreads();
  const int lead = lead_s;
  const bool same = share_agrees(a, b, lead, d, tid, kShareThreads);
  if (__syncthreads_or(same ? 0 : 1)) {
    if (tid == 0) a.joined[b] = -1;
  } else if (tid == 0) {
    a.joined[b] = lead;
  }
}

__global__ __launch_bounds__(kPackThreads) void share_pack_kernel(
    ShareArgs a, int with_rows) {
  __shared__ PackLds s;
  share_pack(a, s, with_rows != 0);
}

__global__ __launch_bounds__(256) void share_rows_kernel(ShareArgs a) {
  const int b = blockIdx.x, i = blockIdx.y * 256 + threadIdx.x;
  const int2 group = a.view.group_of[b];
  const int4 rq = a.view.req[b];
  if (group.x >= 0 && i <= rq.y)
    a.view.rows[group.y + rq.w + i] = b * (a.g.N + 1) + i;
}

// Small tables: one workgroup does all of it, then a wave a request.
constexpr int kSmallBatch = 64;
constexpr int kSmallTable = 16384;   // table entries, and
constexpr int kPackRows = 16384;     // rows that one workgroup goes through
// Comparisons of entries that one workgroup makes at most: 43 requests of 79
// entries 13.7 us, 42 of 207 23.7 and 17 in four launches.
constexpr int64_t kSmallWork = 1 << 17;

__global__ __launch_bounds__(kPackThreads) void share_small_kernel(
    ShareArgs a) {
  __shared__ PackLds s;
  __shared__ unsigned long long best_s[kSmallBatch];
  __shared__ int full_s[kSmallBatch], place_s[kSmallBatch];
  __shared__ int col[kSmallTable];
  const int tid = threadIdx.x, lane = tid & 63;
  int most = 0;
  if (tid < a.g.batch) {
    best_s[tid] = 0;
    full_s[tid] = most = share_pages(a, tid);
  }
  __syncthreads();
  for (int b = 0; b < a.g.batch; ++b) most = max(most, full_s[b]);
  // all places at once, or as many as there is room and threads for
  int wide = 0;
  while (1 << wide < most && 2 << wide <= kPackThreads &&
         a.g.batch << (wide + 1) <= kSmallTable)
    ++wide;
  for (int j0 = 0; j0 < most; j0 += 1 << wide)
    if (a.g.batch << wide <= 4 * kPackThreads)
      share_columns<2>(a, j0, wide, full_s, col, best_s);
    else
      share_columns<8>(a, j0, wide, full_s, col, best_s);
  __syncthreads();
  if (tid < a.g.batch) a.place[tid] = place_s[tid] = share_place(a, best_s[tid]);
  __syncthreads();
  for (int b = tid >> 6; b < a.g.batch; b += kPackThreads / kWave) {
    const int d = place_s[b];
    int lead = -1;
    if (d >= 0) {
      lead = share_lead(a, b, d, place_s, lane, kWave);
      lead = -wave_max(-lead);
      if (__ballot(!share_agrees(a, b, lead, d, lane, kWave))) lead = -1;
    }
    if (lane == 0) a.joined[b] = lead;
  }
  __syncthreads();
  share_pack(a, s, true);
}

}  // namespace

int share_blocks(const pct_cache_shape& sh) {
  const int64_t x = ((int64_t)sh.max_pages + (1 << kWide) - 1) >> kWide;
  return (int)(x < kShareBlocks ? x : kShareBlocks);
}

hipError_t launch_share(const ShareArgs& a, hipStream_t s) {
  const PageGeom& g = a.g;
  const int64_t rows = (int64_t)g.batch * (g.N + 1);
  const int64_t entries = (int64_t)g.batch * g.max_pages;
  if (g.batch <= kSmallBatch && entries <= kSmallTable &&
      entries * g.batch <= kSmallWork && rows <= kPackRows) {
    hipLaunchKernelGGL(share_small_kernel, dim3(1), dim3(kPackThreads), 0, s,
                       a);
    return hipGetLastError();
  }
  const size_t lds = (size_t)g.batch * (12 + (4 << kWide));
  // (few requests: two entries of a thread)
  const bool few = g.batch <= 2 * (kShareThreads >> kWide);
  const auto kernel = few ? share_columns_kernel<2> : share_columns_kernel<8>;
  hipLaunchKernelGGL(kernel, dim3(a.blocks), dim3(kShareThreads), lds, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(share_pick_kernel, dim3(g.batch), dim3(kWave), 0, s, a,
                     a.blocks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(share_join_kernel, dim3(g.batch), dim3(kShareThreads), 0,
                     s, a);
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
