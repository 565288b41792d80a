// k_pages.hip -- pages that several requests hold: places freed and trimmed
// with counts of holders, contexts forked into other places, and the pages in
// use moved to the front of the cache.
//
// extra[p] counts the holders of page p beyond its first.  A holder that lets
// go subtracts one; below zero nobody holds the page any more.  Which holder
// was the last is a matter of timing, so pages do not go to the ring from
// there: a second pass goes through the counts and appends the pages below
// zero in ascending order.
//
// Small calls are chains of dependent loads: 4 places of 63 pages freed 3.8
// us, forked again 4.1 (the plan) and 4.0 (table rows and the rows of 32
// layers).  The copies are bound by memory: 64 forks of 31 rows at most in 16
// layers 9.3 us for 43 MB; a compaction that moves 1.44 GB 529 us, 5.4 TB/s
// read and written (a copy of 1 GiB reaches 5.06).
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

namespace {

constexpr int kThreads = 1024;        // of the kernels of one workgroup
constexpr int kSeg = 16 * kThreads;   // pages of a workgroup of a scan
constexpr int kSmallPlaces = 64;      // places that one workgroup goes through

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A value that other waves of this workgroup may have written before a
// barrier: read past the L1, as atomics write.  (The barrier orders what one
// workgroup does; fences for the whole GPU write back the L2, 2 .. 5 us each.)
__device__ __forceinline__ int fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ int wrap(int64_t x, int n) {
  return (int)(x - (x / n) * n);
}

__device__ __forceinline__ int clamp_held(int h, int max_pages) {
  return min(max(h, 0), max_pages);
}

// ring head and count as the calls take them
__device__ __forceinline__ int2 ring_now(const PagesArgs& a) {
  int head = a.ring_state[0] % a.g.n_pages;
  head += head < 0 ? a.g.n_pages : 0;
  return make_int2(head, min(max(a.ring_state[1], 0), a.g.n_pages));
}

// exclusive prefix sum over the workgroup, and the sum
__device__ __forceinline__ int block_prefix(int x, int* wave_sum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += y;
  }
  __syncthreads();
  if (lane == kWave - 1) wave_sum[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    before += w < wave ? wave_sum[w] : 0;
    all += wave_sum[w];
  }
  total = all;
  return before + incl - x;
}

// Pages of a segment as bits: wave w has the pages from w * 1024 on, bit `lane`
// of word e is page 64 e + lane of them.  USED: pages that are held (extra not
// below zero), else those that are not.
struct Bits {
  uint64_t word[16];
  int count;  // of the wave
};
__device__ __forceinline__ int wave_page(int seg) {
  return seg * kSeg +
         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (16 * kWave);
}
template <bool USED, typename Read>
__device__ __forceinline__ Bits segment_bits(const PagesArgs& a, int seg,
                                             Read read) {
  const int lane = threadIdx.x & 63, P = a.g.n_pages, p0 = wave_page(seg);
  Bits x;
  x.count = 0;
  int v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    v[e] = read(min(p0 + e * kWave + lane, P - 1));
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int p = p0 + e * kWave + lane;
    x.word[e] = __ballot(p < P && (USED ? v[e] >= 0 : v[e] < 0));
    x.count += __popcll(x.word[e]);
  }
  return x;
}
template <bool USED>
__device__ __forceinline__ Bits segment_bits(const PagesArgs& a, int seg) {
  return segment_bits<USED>(a, seg, [&](int p) { return fresh(a.extra + p); });
}
// set bits of a word below this lane's
__device__ __forceinline__ int bits_before(uint64_t word) {
  return __builtin_amdgcn_mbcnt_hi(
      (uint32_t)(word >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)word, 0));
}

// Sum of the waves' x before this one, and of all.
__device__ __forceinline__ int waves_prefix(int x, int* wave_sum, int& total) {
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) wave_sum[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kThreads / kWave; ++w) {
    const int y = wave_sum[w];
    before += w < wave ? y : 0;
    total += y;
  }
  return before;
}

// The pages [keep, held) of request b let go, by `threads` threads.
__device__ __forceinline__ void let_go(const PagesArgs& a, int b, int keep,
                                       int held, int t, int threads) {
  int32_t* table = a.table + (int64_t)b * a.g.max_pages;
  for (int j = keep + t; j < held; j += threads) {
    const int p = table[j];
    if ((unsigned)p < (unsigned)a.g.n_pages) atomicSub(&a.extra[p], 1);
    table[j] = -1;
  }
}

// Place i of the call: its request (-1: none), and the pages it keeps and
// held.  One lane asks.
__device__ __forceinline__ int place_of(const PagesArgs& a, int i, int& keep,
                                        int& held) {
  const PageGeom& g = a.g;
  keep = held = 0;
  if (a.places) {
    const int b = a.places[i];
    if (b < 0 || b >= g.batch) return -1;
    // (a place that is named twice is emptied once)
    held = clamp_held(atomicExch(&a.held[b], 0), g.max_pages);
    a.ctx[b] = 0;
    return b;
  }
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[i], g.N) : g.N;
  const int64_t need =
      ((int64_t)clamp_ctx(a.ctx[i]) + n + (1 << g.shift)) >> g.shift;
  held = clamp_held(a.held[i], g.max_pages);
  keep = (int)min(need, (int64_t)held);
  if (keep < held) a.held[i] = keep;
  return i;
}

// Appends the pages of segment seg that nobody holds any more to the ring,
// after `before` others; returns how many.
__device__ __forceinline__ int append_segment(const PagesArgs& a, int seg,
                                              int2 ring, int before,
                                              int* wave_sum) {
  const Bits gone = segment_bits<false>(a, seg);
  const int lane = threadIdx.x & 63, p0 = wave_page(seg);
  int total;
  int at = before + waves_prefix(gone.count, wave_sum, total);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if (gone.word[e] == 0) continue;
    if ((gone.word[e] >> lane) & 1) {
      const int p = p0 + e * kWave + lane;
      a.ring[wrap((int64_t)ring.x + ring.y + at + bits_before(gone.word[e]),
                  a.g.n_pages)] = p;
      a.extra[p] = 0;
    }
    at += __popcll(gone.word[e]);
  }
  return total;
}

// few places and pages: everything in one workgroup
__global__ __launch_bounds__(kThreads) void release_small_kernel(PagesArgs a) {
  __shared__ int wave_sum[kThreads / kWave];
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < a.m; i += kThreads / kWave) {
    int b = 0, keep = 0, held = 0;
    if (lane == 0) b = place_of(a, i, keep, held);
    b = __builtin_amdgcn_readfirstlane(b);
    keep = __builtin_amdgcn_readfirstlane(keep);
    held = __builtin_amdgcn_readfirstlane(held);
    if (b >= 0) let_go(a, b, keep, held, lane, kWave);
  }
  const int2 ring = ring_now(a);
  __syncthreads();
  const int more = append_segment(a, 0, ring, 0, wave_sum);
  if (threadIdx.x == 0) {
    a.ring_state[0] = ring.x;
    a.ring_state[1] = min(ring.y + more, a.g.n_pages);
  }
}

__global__ __launch_bounds__(256) void release_kernel(PagesArgs a) {
  __shared__ int s[3];
  if (threadIdx.x == 0) s[0] = place_of(a, blockIdx.x, s[1], s[2]);
  __syncthreads();
  if (s[0] >= 0) let_go(a, s[0], s[1], s[2], threadIdx.x, 256);
}

// count[seg]: pages of a segment that nobody holds any more; the ring's state
// of before behind the counts
__global__ __launch_bounds__(kThreads) void released_count_kernel(PagesArgs a,
                                                                  int segs) {
  __shared__ int wave_sum[kThreads / kWave];
  int total;
  waves_prefix(segment_bits<false>(a, blockIdx.x).count, wave_sum, total);
  if (threadIdx.x != 0) return;
  a.count[blockIdx.x] = total;
  if (blockIdx.x == 0) {
    const int2 ring = ring_now(a);
    a.count[segs] = ring.x;
    a.count[segs + 1] = ring.y;
  }
}

// sum of count[from .. to), by the whole workgroup
__device__ __forceinline__ int sum_counts(const int32_t* count, int from,
                                          int to, int* wave_sum) {
  int n = 0, total;
  for (int i = from + threadIdx.x; i < to; i += blockDim.x) n += count[i];
  block_prefix(n, wave_sum, total);
  return total;
}

__global__ __launch_bounds__(kThreads) void released_append_kernel(
    PagesArgs a, int segs) {
  __shared__ int wave_sum[kThreads / kWave];
  const int seg = blockIdx.x;
  // (one segment: nothing was counted, nobody else reads the state)
  const int2 ring = segs == 1 ? ring_now(a)
                              : make_int2(a.count[segs], a.count[segs + 1]);
  const int before = sum_counts(a.count, 0, seg, wave_sum);
  const int mine = append_segment(a, seg, ring, before, wave_sum);
  if (seg == segs - 1 && threadIdx.x == 0) {
    a.ring_state[0] = ring.x;
    a.ring_state[1] = min(ring.y + before + mine, a.g.n_pages);
  }
}

// ---------------------------------------------------------------------
// Forks.  One workgroup decides all pairs on the state of before the call and
// gives out the pages for the parts of pages, in the order of the pairs;
// then a workgroup per pair writes its table row and counts, and others copy
// the rows of its last page.
constexpr int kClaims = 4096;  // places whose claims are kept in LDS

__global__ __launch_bounds__(kThreads) void fork_plan_kernel(ForkArgs f) {
  __shared__ int wave_sum[kThreads / kWave];
  __shared__ int s_taken, claim_s[kClaims];
  const PagesArgs& a = f.a;
  const PageGeom& g = a.g;
  const int tid = threadIdx.x, P = g.n_pages;
  const bool in_lds = g.batch <= kClaims;
  const auto place = [&](int b) { return b >= 0 && b < g.batch; };
  const int2 ring = ring_now(a);
  if (tid == 0) s_taken = 0;
  // the first pair that names a place has it
  for (int i = tid; i < a.m; i += kThreads) {
    const int d = f.dst[i];
    if (place(d)) {
      if (in_lds)
        claim_s[d] = a.m;
      else
        f.claim[d] = a.m;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.m; i += kThreads) {
    const int d = f.dst[i];
    if (place(d)) {
      if (in_lds)
        atomicMin(&claim_s[d], i);
      else
        atomicMin(&f.claim[d], i);
    }
  }
  __syncthreads();
  int base = 0;
  for (int i0 = 0; i0 < a.m; i0 += kThreads) {
    const int i = i0 + tid;
    bool ok = false;
    int s = 0, d = 0, len = 0, need = 0, rest = 0;
    if (i < a.m) {
      s = f.src[i];
      d = f.dst[i];
      ok = place(s) && place(d) && s != d;
    }
    if (ok) {
      len = clamp_ctx(a.ctx[s]);
      if (f.length) len = min(len, max(f.length[i], 0));
      rest = len & ((1 << g.shift) - 1);
      need = (len >> g.shift) + (rest > 0 ? 1 : 0);
      ok = (in_lds ? claim_s[d] : fresh(f.claim + d)) == i &&
           a.held[d] <= 0 && need <= clamp_held(a.held[s], g.max_pages);
      if (ok && rest > 0)
        ok = (unsigned)a.table[(int64_t)s * g.max_pages + need - 1] <
             (unsigned)P;
    }
    int total;
    const int at = base + block_prefix(ok && rest > 0, wave_sum, total);
    base += total;
    // from the first that gets no page on, none does
    if (ok && rest > 0) {
      ok = at < ring.y;
      if (ok) atomicMax(&s_taken, at + 1);
    }
    if (i < a.m) {
      f.req[i] = make_int4(
          ok ? s : -1, d, len,
          ok && rest > 0 ? a.ring[wrap((int64_t)ring.x + at, P)] : -1);
      f.done[i] = ok ? 1 : 0;
    }
  }
  __syncthreads();
  // the state, once every pair has been decided on the one of before
  for (int i = tid; i < a.m; i += kThreads) {
    const int4 rq = f.req[i];
    if (rq.x < 0) continue;
    a.ctx[rq.y] = rq.z;
    a.held[rq.y] = (int)(((int64_t)rq.z + (1 << g.shift) - 1) >> g.shift);
  }
  if (tid == 0) {
    a.ring_state[0] = wrap((int64_t)ring.x + s_taken, P);
    a.ring_state[1] = ring.y - s_taken;
  }
}

// A wave copies the rows of one (layer, cache, head); grid (pairs, groups of
// 4 waves, pieces of the rows).
__global__ __launch_bounds__(256) void fork_apply_kernel(ForkArgs f,
                                                         int runs) {
  const PagesArgs& a = f.a;
  const PageGeom& g = a.g;
  const int4 rq = f.req[blockIdx.x];
  if (rq.x < 0) return;
  const int tid = threadIdx.x;
  const int full = rq.z >> g.shift, rest = rq.z & ((1 << g.shift) - 1);
  const int32_t* from = a.table + (int64_t)rq.x * g.max_pages;
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    int32_t* to = a.table + (int64_t)rq.y * g.max_pages;
    for (int j = tid; j < full; j += 256) {
      const int p = from[j];
      to[j] = p;
      if ((unsigned)p < (unsigned)g.n_pages) atomicAdd(&a.extra[p], 1);
    }
    if (rest > 0 && tid == 0) to[full] = rq.w;
  }
  if (rest == 0 || (unsigned)rq.w >= (unsigned)g.n_pages) return;
  const int hc = g.D / 8;
  const int64_t page_chunks = ((int64_t)g.Hkv << g.shift) * hc;
  const int n = rest * hc, step = 64 * gridDim.z;
  const int64_t from_page = from[full];
  for (int run = blockIdx.y * 4 + (tid >> 6); run < runs;
       run += 4 * gridDim.y) {
    const int h = run % g.Hkv, lk = run / g.Hkv;
    uint4* cache = ((lk & 1) ? a.vc : a.kc) +
                   (int64_t)(lk >> 1) * a.layer_stride +
                   ((int64_t)h << g.shift) * hc;
    const u32x4* src =
        reinterpret_cast<const u32x4*>(cache + from_page * page_chunks);
    u32x4* dst = reinterpret_cast<u32x4*>(cache + rq.w * page_chunks);
    for (int i = blockIdx.z * 64 + (tid & 63); i < n; i += 4 * step) {
      u32x4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e * step < n) x[e] = src[i + e * step];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e * step < n) dst[i + e * step] = x[e];
    }
  }
}

// ---------------------------------------------------------------------
// Compaction.  With the holders counted (extra: holders - 1), T pages are in
// use.  The used pages from T on, in ascending order, move to the unused ones
// below T, in ascending order: as many of the one as of the other, and no
// page is both read and written.
// extra: a.extra, or a copy in LDS
__device__ __forceinline__ void count_pages(const PagesArgs& a, int32_t* extra,
                                            int b, int t, int threads) {
  const int held = clamp_held(a.held[b], a.g.max_pages);
  const int32_t* table = a.table + (int64_t)b * a.g.max_pages;
  for (int j = t; j < held; j += threads) {
    const int p = table[j];
    if ((unsigned)p < (unsigned)a.g.n_pages) atomicAdd(&extra[p], 1);
  }
}

// Lists the moves of a segment: `before` used pages precede it, `total` are
// in use, of which `low` below page `total`.
__device__ __forceinline__ void list_moves(const CompactArgs& c,
                                           const Bits& used, int seg,
                                           int before, int total, int low,
                                           int* wave_sum) {
  const PagesArgs& a = c.a;
  const int lane = threadIdx.x & 63, p0 = wave_page(seg);
  int sum;
  int at = before + waves_prefix(used.count, wave_sum, sum);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int p = p0 + e * kWave + lane;
    const int u = at + bits_before(used.word[e]);
    at += __popcll(used.word[e]);
    if (p >= a.g.n_pages) continue;
    const bool on = (used.word[e] >> lane) & 1;
    if (!on && p < total) c.hole[p - u] = p;
    if (on && p >= total) {
      c.high[u - low] = p;
      c.rank[p] = u - low;
    }
    // the ring: the pages behind those in use
    a.ring[p] = wrap((int64_t)total + p, a.g.n_pages);
  }
  if (seg == 0 && threadIdx.x == 0) {
    a.ring_state[0] = 0;
    a.ring_state[1] = a.g.n_pages - total;
    c.info[0] = total;
    c.info[1] = total - low;
  }
}

// used pages of a segment below page `end`
__device__ __forceinline__ int used_below(const Bits& used, int seg, int end,
                                          int* wave_sum) {
  const int p0 = wave_page(seg);
  int n = 0, sum;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int left = end - p0 - e * kWave;
    const uint64_t mask =
        left <= 0 ? 0 : left >= 64 ? ~0ull : (1ull << left) - 1;
    n += __popcll(used.word[e] & mask);
  }
  waves_prefix(n, wave_sum, sum);
  return sum;
}

__global__ __launch_bounds__(kThreads) void compact_small_kernel(
    CompactArgs c) {
  __shared__ int wave_sum[kThreads / kWave];
  __shared__ int32_t extra[kSeg];
  const PagesArgs& a = c.a;
  const int P = a.g.n_pages;
  for (int p = threadIdx.x; p < P; p += kThreads) extra[p] = -1;
  __syncthreads();
  for (int b = threadIdx.x >> 6; b < a.g.batch; b += kThreads / kWave)
    count_pages(a, extra, b, threadIdx.x & 63, kWave);
  __syncthreads();
  const Bits used =
      segment_bits<true>(a, 0, [&](int p) { return extra[p]; });
  const int total = used_below(used, 0, P, wave_sum);
  const int low = used_below(used, 0, total, wave_sum);
  list_moves(c, used, 0, 0, total, low, wave_sum);
  for (int p = threadIdx.x; p < P; p += kThreads) a.extra[p] = extra[p];
}

__global__ __launch_bounds__(256) void compact_clear_kernel(PagesArgs a) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p < a.g.n_pages) a.extra[p] = -1;
}

__global__ __launch_bounds__(256) void compact_holders_kernel(PagesArgs a) {
  count_pages(a, a.extra, blockIdx.x, threadIdx.x, 256);
}

__global__ __launch_bounds__(kThreads) void compact_count_kernel(
    CompactArgs c) {
  __shared__ int wave_sum[kThreads / kWave];
  const int n = used_below(segment_bits<true>(c.a, blockIdx.x), blockIdx.x,
                           c.a.g.n_pages, wave_sum);
  if (threadIdx.x == 0) c.a.count[blockIdx.x] = n;
}

__global__ __launch_bounds__(kThreads) void compact_list_kernel(CompactArgs c) {
  __shared__ int wave_sum[kThreads / kWave];
  const int segs = gridDim.x, seg = blockIdx.x;
  const int total = sum_counts(c.a.count, 0, segs, wave_sum);
  const int edge = min(total / kSeg, segs - 1);  // its segment of page `total`
  const int low = sum_counts(c.a.count, 0, edge, wave_sum) +
                  used_below(segment_bits<true>(c.a, edge), edge, total,
                             wave_sum);
  const int before = sum_counts(c.a.count, 0, seg, wave_sum);
  list_moves(c, segment_bits<true>(c.a, seg), seg, before, total, low,
             wave_sum);
}

// Tables, holders and the pages themselves.  The first workgroups rewrite a
// table row each and the counts; the others copy pages, a workgroup a piece
// of kPiece chunks at a time.
constexpr int kPiece = 1024;

__global__ __launch_bounds__(256) void compact_apply_kernel(CompactArgs c,
                                                            int rows,
                                                            int pieces) {
  const PagesArgs& a = c.a;
  const PageGeom& g = a.g;
  const int tid = threadIdx.x;
  const int total = c.info[0], moves = c.info[1];
  if ((int)blockIdx.x < rows) {
    const int b = blockIdx.x;
    const int held = clamp_held(a.held[b], g.max_pages);
    const int32_t* from = a.table + (int64_t)b * g.max_pages;
    int32_t* to = c.table_out + (int64_t)b * g.max_pages;
    for (int j = tid; j < g.max_pages; j += 256) {
      int p = from[j];
      if (j < held && p >= total && p < g.n_pages) p = c.hole[c.rank[p]];
      to[j] = p;
    }
    for (int64_t p = (int64_t)total + b * 256 + tid; p < g.n_pages;
         p += (int64_t)rows * 256) {
      const int e = a.extra[p];
      if (e >= 0) a.extra[c.hole[c.rank[p]]] = e;
      a.extra[p] = 0;
    }
    return;
  }
  const int64_t page_chunks = ((int64_t)g.Hkv << g.shift) * (g.D / 8);
  const int64_t per_move = (int64_t)a.layers * 2 * pieces;
  for (int64_t x = blockIdx.x - rows; x < moves * per_move;
       x += gridDim.x - rows) {
    const int k = (int)(x / per_move);
    const int y = (int)(x - k * per_move);
    const int lk = y / pieces, piece = y - lk * pieces;
    uint4* cache =
        ((lk & 1) ? a.vc : a.kc) + (int64_t)(lk >> 1) * a.layer_stride;
    const u32x4* src =
        reinterpret_cast<const u32x4*>(cache + c.high[k] * page_chunks);
    u32x4* dst = reinterpret_cast<u32x4*>(cache + c.hole[k] * page_chunks);
    const int64_t i = (int64_t)piece * kPiece + tid;
    u32x4 v[kPiece / 256];
#pragma unroll
    for (int e = 0; e < kPiece / 256; ++e)
      if (i + e * 256 < page_chunks) v[e] = src[i + e * 256];
#pragma unroll
    for (int e = 0; e < kPiece / 256; ++e)
      if (i + e * 256 < page_chunks) dst[i + e * 256] = v[e];
  }
}

int segments(int n_pages) { return (int)(((int64_t)n_pages + kSeg - 1) / kSeg); }

}  // namespace

size_t release_workspace(const pct_cache_shape& sh) {
  return ((size_t)segments(sh.n_pages) + 2) * sizeof(int32_t);
}

hipError_t launch_release(const PagesArgs& a, hipStream_t s) {
  if (a.m <= kSmallPlaces && a.g.n_pages <= kSeg) {
    hipLaunchKernelGGL(release_small_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const int segs = segments(a.g.n_pages);
  hipLaunchKernelGGL(release_kernel, dim3(a.m), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (segs > 1) {
    hipLaunchKernelGGL(released_count_kernel, dim3(segs), dim3(kThreads), 0, s,
                       a, segs);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(released_append_kernel, dim3(segs), dim3(kThreads), 0, s,
                     a, segs);
  return hipGetLastError();
}

hipError_t launch_fork(const ForkArgs& f, hipStream_t s) {
  const PageGeom& g = f.a.g;
  hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(kThreads), 0, s, f);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int runs = f.a.layers * 2 * g.Hkv;
  const int chunks = (g.D / 8) << g.shift;
  const int z = chunks <= 512 ? 1 : chunks / 512 < 16 ? chunks / 512 : 16;
  const int y = runs < 4 * 65535 ? (runs + 3) / 4 : 65535;
  hipLaunchKernelGGL(fork_apply_kernel, dim3(f.a.m, y, z), dim3(256), 0, s, f,
                     runs);
  return hipGetLastError();
}

size_t compact_workspace(const pct_cache_shape& sh) {
  return ((size_t)segments(sh.n_pages) + 4 + 3 * (size_t)sh.n_pages) *
         sizeof(int32_t);
}

hipError_t launch_compact(const CompactArgs& c, hipStream_t s) {
  const PagesArgs& a = c.a;
  const PageGeom& g = a.g;
  hipError_t e;
  if (g.batch <= kSmallPlaces && g.n_pages <= kSeg) {
    hipLaunchKernelGGL(compact_small_kernel, dim3(1), dim3(kThreads), 0, s, c);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else {
    const int segs = segments(g.n_pages);
    hipLaunchKernelGGL(compact_clear_kernel,
                       dim3((unsigned)(((int64_t)g.n_pages + 255) / 256)),
                       dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_holders_kernel, dim3(g.batch), dim3(256), 0, s,
                       a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_count_kernel, dim3(segs), dim3(kThreads), 0, s,
                       c);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(compact_list_kernel, dim3(segs), dim3(kThreads), 0, s,
                       c);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t page_chunks = ((int64_t)g.Hkv << g.shift) * (g.D / 8);
  const int pieces = (int)((page_chunks + kPiece - 1) / kPiece);
  // at most half of the pages move
  const int64_t work = ((int64_t)g.n_pages + 1) / 2 * a.layers * 2 * pieces;
  const int copies = (int)(work < 4096 ? work : 4096);
  hipLaunchKernelGGL(compact_apply_kernel, dim3(g.batch + copies), dim3(256),
                     0, s, c, g.batch, pieces);
  return hipGetLastError();
}

}  // namespace pct
