// k_attend_impl.h -- softmax attention of a round's rows over a paged
// key-value cache, on MFMA.  For a row with the seen positions S,
//   out = sum_{t in S} p_t v_t / sum_{t in S} p_t,  p_t = 2^(z_t - m),
//   z_t = |scale| log2(e) (+-q . k_t),  lse = ln(2) (m + log2 sum p_t),
// in one pass over the positions.  m only has to be near the largest z_t: it
// is raised (and the sums so far are scaled down) when a z_t comes that is
// more than kRaise above it, so p stays below 2^kRaise and most tiles need
// neither a reduction over lanes nor a rescaling.  p is rounded to the cache's
// type for the second product (the sums of p and of p v are fp32), which
// bf16 does to 2^-8 of every p.  fp16 rounds p below 2^-14 to its least step
// 2^-24 instead, and p below 2^-25 to nothing, while they all count in the
// sum: 32 k keys at 2^-25 of the largest are 2^-10 of the result.  It holds
// 2^kLift p instead (at most 2^(kRaise + kLift) = 2^15; the largest fp16 is just below
// 2^16), and its sums are 2^kLift times as large until they are divided.
//
// Both products are computed transposed, with v_mfma_f32_16x16x32:
//   S^T[key][row] = K Q^T     A = 16 keys of the tile, B = 16 query rows
//   O^T[d][row]  += V^T P^T   A = 16 elements of 32 keys, B = P
// so a lane owns one row of the query tile (column lane % 16) in S, P and O,
// and the fp32 scores of two 16-key blocks, rounded, are already the B
// operand of the second product: its k index (lane / 16, e) stands for key
// 4 (lane / 16) + e of the first block (e < 4) or of the second.  The A
// operand of V^T in that order comes from row-major V by transposing LDS
// reads (ds_read_b64_tr_b16: 4 keys of one element per lane).
//
// The query rows of one key-value head are packed (row i, head g of the
// group) -> i G + g.  Up to 16 of them are the columns of every wave, whose
// waves take different keys (k_attend_rows.h, bound by memory); more are cut
// into tiles whose waves share the keys (k_attend_tiles.h, bound by the
// matrix units and the exponentials).
//
// Work is the list of all (request, head, row tile, step of KS keys), cut
// into contiguous runs of equal work, one per workgroup, whatever the lengths
// of the requests (known on the device only).  A row tile whose steps lie in
// one run is finished there; otherwise each run leaves its unnormalised
// sums in the workspace and the join kernel adds them up in order of runs,
// so results do not depend on timing.
#pragma once
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr float kRaise = 8.f;

template <bool BF16>
__device__ __forceinline__ f32x4 mfma16(s16x8 x, s16x8 y, f32x4 c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0,
        0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(
        __builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0,
        0);
}

// eight floats rounded to the element type (to nearest even)
template <bool BF16>
__device__ __forceinline__ s16x8 round8(f32x8 x) {
  if constexpr (BF16)
    return __builtin_bit_cast(s16x8, __builtin_convertvector(x, bf16x8));
  else
    return __builtin_bit_cast(s16x8, __builtin_convertvector(x, f16x8));
}

// four floats rounded to the element type
template <bool BF16>
__device__ __forceinline__ uint2 round4(f32x4 x) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  if constexpr (BF16)
    return __builtin_bit_cast(uint2, __builtin_convertvector(x, bf16x4));
  else
    return __builtin_bit_cast(uint2, __builtin_convertvector(x, f16x4));
}

template <bool BF16>
__device__ __forceinline__ float elem(uint16_t b) {
  if constexpr (BF16) return bf16_bits_to_float(b);
  return (float)__builtin_bit_cast(_Float16, b);
}

// Max and sum over the four lanes that hold one row (lane % 16): a swap of
// x with a copy of itself leaves both partners' values in every lane.
template <typename Op>
__device__ __forceinline__ float row_reduce(float x, Op op) {
  int u = __builtin_bit_cast(int, x);
  auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  int y = (int)p[0], z = (int)p[1];
  x = op(__builtin_bit_cast(float, y), __builtin_bit_cast(float, z));
  u = __builtin_bit_cast(int, x);
  p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  y = (int)p[0];
  z = (int)p[1];
  return op(__builtin_bit_cast(float, y), __builtin_bit_cast(float, z));
}
__device__ __forceinline__ float row_max(float x) {
  return row_reduce(x, [](float p, float q) { return fmaxf(p, q); });
}
__device__ __forceinline__ float row_sum(float x) {
  return row_reduce(x, [](float p, float q) { return p + q; });
}

// x as a value that the compiler cannot trace: what is derived from it inside
// a loop is computed there instead of held in registers across the loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// x of lane l
__device__ __forceinline__ uint64_t shfl_bits(uint64_t x, int l) {
  const uint32_t lo = __shfl((int)(uint32_t)x, l, kWave);
  const uint32_t hi = __shfl((int)(x >> 32), l, kWave);
  return (uint64_t)hi << 32 | lo;
}

// the lowest n bits (n clamped to [0, 64])
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : (n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1);
}

// Work of one request in units: a step of a row tile.
struct AttendReq {
  int ctx, n, L;   // context, nodes, positions
  int M, RT, KT;   // packed rows, row tiles, steps of a row tile
  int64_t units;   // of all heads and row tiles
};
template <int MT, int KS>
__device__ __forceinline__ AttendReq attend_lengths(const AttendArgs& a,
                                                    int ctx, int n) {
  AttendReq r;
  // A context that does not fit the block table ends with it: its last
  // position stands in for the root, and the nodes are past the end.
  const int cap = a.g.max_pages << a.g.shift;
  r.n = n;
  r.ctx = min(ctx, cap - 1);
  r.L = min(r.ctx + n + 1, cap);
  r.M = (n + 1) * a.G;
  r.RT = (r.M + MT - 1) / MT;
  r.KT = (r.L + KS - 1) / KS;
  r.units = (int64_t)a.g.Hkv * r.RT * r.KT;
  return r;
}
// Lengths of request b; uniform: b is the same in every lane, and the lengths
// are held in scalar registers.
template <int MT, int KS>
__device__ __forceinline__ AttendReq attend_req(const AttendArgs& a, int b,
                                                bool uniform = false) {
  const PageGeom& g = a.g;
  int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  int ctx = clamp_ctx(g.ctx_len[b]);
  if (uniform) {
    n = __builtin_amdgcn_readfirstlane(n);
    ctx = __builtin_amdgcn_readfirstlane(ctx);
  }
  return attend_lengths<MT, KS>(a, ctx, n);
}

// a 64-bit value of lane l
__device__ __forceinline__ int64_t lane_value(int64_t x, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, l);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(x >> 32), l);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// x / d for x >= 0, d > 0, which mostly fit 32 bits.
__device__ __forceinline__ int64_t div_up_to_64(int64_t x, int64_t d) {
  if (((x | d) >> 31) == 0) return (uint32_t)x / (uint32_t)d;
  return x / d;
}

// How many runs `units` units of row tiles of mostly `steps` steps are cut
// into.  Up to kWhole steps of shared tiles stay together: the sums that the
// runs of a row tile leave, and their join, would cost more (2 requests of
// 256 rows over 306 positions: 26 us, cut at 4 of their 5 steps 33).  Longer
// row tiles are cut finely while every run has a CU of its own, and less so
// beyond that: two runs on a CU slow each other down.
template <int FEW, int LEAST>
__device__ __forceinline__ int64_t runs_for(int64_t units, int steps) {
  const bool whole = steps <= kWhole && LEAST > 1;
  const int few = whole ? steps : FEW, many = whole ? steps : LEAST;
  const int64_t x = div_up_to_64(units + few - 1, few);
  const int64_t y = div_up_to_64(units, many);
  return min(x, max(y, (int64_t)kCus));
}

// How the work is cut into runs, one per workgroup.
//
// Lines: the units of all requests in the order (request, head, row tile,
// step), cut into runs of equal length.  Any batch.
//
// Levels: where all requests have the same number of row tiles, level i is
// row tile i of every head in the order (request, head, step).  All levels
// are cut at the same places into blocks, and the runs of one block, one per
// level, are on one XCD: they read the same keys at the same time, so the
// keys come from its L2 for all levels but the first.  With lines a run
// goes through the row tiles of a head one after the other, and each of
// them reads the keys from memory again.
struct AttendRun {
  int run;  // index of this run; a row tile's runs follow each other
  int64_t u, end;
  int b;          // request that holds u; its units begin at b_off
  int64_t b_off;
  int level;      // row tile of the run, -1: lines
  // Run (block) j of `blocks` begins at unit floor(j total / blocks): as many
  // runs for every row tile of equal lengths end where it ends.
  int blocks;
  int64_t total;
  __device__ __forceinline__ int64_t start(int j) const {
    return div_up_to_64(j * total, blocks);
  }
  // run that holds unit x of the lines, or of this run's level
  __device__ __forceinline__ int owner(int64_t x) const {
    const int j = (int)div_up_to_64((x + 1) * blocks - 1, total);
    return level < 0 ? j : level * blocks + j;
  }
  __device__ __forceinline__ int64_t units(const AttendArgs& a,
                                           const AttendReq& rq) const {
    return level < 0 ? rq.units
                     : (rq.M > 0 ? (int64_t)a.g.Hkv * rq.KT : (int64_t)0);
  }
};

// The steps [k0, k1) of head h and row tile rt that a run has from unit u on;
// s0: the row tile's first unit.
struct AttendPiece {
  int h, rt, k0, k1;
  int64_t s0;
};
__device__ __forceinline__ AttendPiece attend_piece(const AttendReq& rq,
                                                    const AttendRun& run) {
  AttendPiece p;
  const int64_t in = run.u - run.b_off;
  const int seg = (int)div_up_to_64(in, rq.KT);
  p.k0 = (int)(in - (int64_t)seg * rq.KT);
  p.k1 = (int)min((int64_t)rq.KT, p.k0 + run.end - run.u);
  p.s0 = run.u - p.k0;
  p.h = run.level < 0 ? seg / rq.RT : seg;
  p.rt = run.level < 0 ? seg - p.h * rq.RT : run.level;
  return p;
}

// Moves on to the request that holds unit u.
template <int MT, int KS>
__device__ __forceinline__ void next_request(const AttendArgs& a,
                                             AttendRun& run, AttendReq& rq) {
  while (run.u >= run.b_off + run.units(a, rq)) {
    run.b_off += run.units(a, rq);
    rq = attend_req<MT, KS>(a, ++run.b, true);
  }
}

// Fills in the run of this workgroup; false when it has none (its entry of
// the join is then empty).  Every wave does this by itself: lane l goes
// through requests l per .. (l + 1) per - 1, and the sums over lanes need no
// LDS.
template <int MT, int KS, int FEW, int LEAST>
__device__ __forceinline__ bool attend_schedule(const AttendArgs& a,
                                                const AttendWs& ws,
                                                AttendRun& r, AttendReq& rq) {
  const PageGeom& g = a.g;
  const int lane = threadIdx.x & 63;
  const int per = (g.batch + 63) / 64;
  const int b0 = lane * per, b1 = min(b0 + per, g.batch);
  int64_t mine = 0, mine1 = 0;  // units of lines, of a level
  int least = 0x7fffffff, most = 0;  // row tiles of a request
  float tiles = 0.f;                 // row tiles of all requests
  AttendReq q{};
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    q = attend_req<MT, KS>(a, b);
    mine += q.units;
    if (q.M > 0) {
      mine1 += (int64_t)g.Hkv * q.KT;
      least = min(least, q.RT);
      most = max(most, q.RT);
      tiles += (float)(g.Hkv * q.RT);
    }
  }
  int64_t incl = mine, incl1 = mine1;
  // (lane `lanes` - 1 is the last one with requests)
  const int lanes = min(g.batch, kWave);
#pragma unroll 1
  for (int d = 1; d < lanes; d <<= 1) {
    const int64_t x = __shfl_up(incl, d, kWave);
    const int64_t y = __shfl_up(incl1, d, kWave);
    if (lane >= d) {
      incl += x;
      incl1 += y;
    }
  }
  const int64_t total = lane_value(incl, lanes - 1);
  const int64_t total1 = lane_value(incl1, lanes - 1);
  const int RT = wave_max(most);
  // steps of a row tile, on average
  const int steps = max(1, (int)((float)total / fmaxf(wave_sum(tiles), 1.f)));
  const bool same = __ballot(least != 0x7fffffff && least != RT) == 0;
  const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
  const int n_wg = gridDim.x, per_xcd = n_wg >> 3;
  // levels, if they keep at least 4 of 5 workgroups busy
  int bx = RT > 0 ? per_xcd / RT : 0;  // blocks of an XCD
  const int fit =
      RT > 0 ? (int)min((int64_t)n_wg, runs_for<FEW, LEAST>(
                                           RT * total1, steps)) / (8 * RT)
             : 0;
  const bool levels = RT > 1 && same && 5 * RT * bx >= 4 * per_xcd && fit > 0;
  bx = min(bx, fit);
  int n_run, xcount;  // runs, and runs of this XCD
  if (levels) {
    n_run = 8 * RT * bx;
    xcount = RT * bx;
    const int j = xcd * bx + at % bx;
    r.level = at / bx;
    r.blocks = 8 * bx;
    r.run = r.level * r.blocks + j;
    r.total = total1;
    r.u = r.start(j);
    r.end = r.start(j + 1);
    incl = incl1;
    mine = mine1;
  } else {
    // neighbouring runs on one XCD (workgroups go round the 8 XCDs)
    n_run = (int)min((int64_t)n_wg, runs_for<FEW, LEAST>(total, steps));
    xcount = (n_run >> 3) + (xcd < (n_run & 7) ? 1 : 0);
    r.level = -1;
    r.run = xcd * (n_run >> 3) + min(xcd, n_run & 7) + at;
    r.blocks = max(n_run, 1);
    r.total = total;
    r.u = r.start(r.run);
    r.end = r.start(r.run + 1);
  }
  if (at >= xcount) {  // no run
    if (ws.row_tiles > 0) return false;
    int before = 0;    // such workgroups of the XCDs before this one
    for (int x = 0; x < xcd; ++x)
      before += per_xcd - (r.level >= 0 ? xcount
                                        : (n_run >> 3) +
                                              (x < (n_run & 7) ? 1 : 0));
    if (threadIdx.x == 0)
      ws.meta[n_run + before + at - xcount] = make_int4(0, 0, 0, -1);
    return false;
  }
  // the lane whose requests hold unit u, then the request
  const int l = __builtin_ctzll(__ballot(r.u < incl));
  r.b = l * per;
  r.b_off = lane_value(incl - mine, l);
  if (per == 1) {
    // (already loaded)
    rq = attend_lengths<MT, KS>(
        a, __builtin_amdgcn_readlane(q.ctx, l),
        __builtin_amdgcn_readlane(q.n, l));
  } else {
    rq = attend_req<MT, KS>(a, r.b, true);
    next_request<MT, KS>(a, r, rq);
  }
  return true;
}

__device__ __forceinline__ void store_meta(const AttendWs& ws, int at,
                                           i32x4 x) {
  reinterpret_cast<i32x4*>(ws.meta)[at] = x;
}

// Notes for the join that the run has the piece pc.
__device__ __forceinline__ void note_piece(const AttendArgs& a,
                                           const AttendWs& ws,
                                           const AttendRun& run,
                                           const AttendReq& rq,
                                           const AttendPiece& pc,
                                           i32x4& join) {
  if (pc.k0 != 0) return;
  // the join adds the runs up to the one that holds the last step
  const int last = pc.k1 < rq.KT ? run.owner(pc.s0 + rq.KT - 1) : -1;
  const i32x4 j = {run.b, pc.h << 20 | pc.rt, run.run, last};
  if (ws.row_tiles == 0)
    join = j;
  else if (threadIdx.x == 0)
    store_meta(ws, (run.b * a.g.Hkv + pc.h) * ws.row_tiles + pc.rt, j);
}

// Query rows m0 + 16 nt + lane % 16 as B operands, as they are;
// irow: their rows (0: the root).
template <class C>
__device__ __forceinline__ void load_queries(const AttendArgs& a, int b, int h,
                                             int m0, int M,
                                             int (&irow)[C::NT],
                                             s16x8 (&qf)[C::NT][C::KSTEP]) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int chd = a.g.D >> 3;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    const int m = m0 + nt * 16 + col;
    const int i = m / a.G;
    irow[nt] = i;
    const bool ok = m < M;
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.q) +
        ((int64_t)b * (a.g.N + 1) + (ok ? i : 0)) * a.qs +
        (h * a.G + (ok ? m - i * a.G : 0)) * a.g.D);
#pragma unroll
    for (int s = 0; s < C::KSTEP; ++s) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok && 4 * s + quad < chd) x = q[4 * s + quad];
      qf[nt][s] = __builtin_bit_cast(s16x8, x);
    }
  }
}

// The scale's sign into the queries; a scale of zero leaves zeros.
template <class C>
__device__ __forceinline__ void sign_queries(const AttendArgs& a,
                                             s16x8 (&qf)[C::NT][C::KSTEP]) {
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int s = 0; s < C::KSTEP; ++s) {
      uint4 x = __builtin_bit_cast(uint4, qf[nt][s]);
      x.x = (x.x & a.qand) ^ a.qxor;
      x.y = (x.y & a.qand) ^ a.qxor;
      x.z = (x.z & a.qand) ^ a.qxor;
      x.w = (x.w & a.qand) ^ a.qxor;
      qf[nt][s] = __builtin_bit_cast(s16x8, x);
    }
}

// The keys t0 .. t0 + 63 that row i of request b sees, as bits (pages and
// the end of the positions aside).
__device__ __forceinline__ uint64_t seen_keys(const AttendArgs& a, int b,
                                              int i, int n, int ctx, int t0) {
  const int j0 = t0 - ctx - 1;       // node of the first key
  uint64_t see = low_bits(-j0);      // the context and the root
  if (i > 0 && i <= n) {
    if (a.mask == nullptr) {
      see |= low_bits(i - j0);
    } else if (j0 > -64) {
      const uint64_t* mr = a.mask + ((int64_t)b * a.g.N + i - 1) * a.words;
      if (j0 < 0) {
        see |= mr[0] << -j0;
      } else {
        const int w = j0 >> 6, sh = j0 & 63;
        if (w < a.words) see |= mr[w] >> sh;
        if (sh != 0 && w + 1 < a.words) see |= mr[w + 1] << (64 - sh);
      }
    }
  }
  return see;
}

// Softmax state of a wave's rows: the reference m of each row (ms: m - kLift,
// 0 while nothing was seen), this lane's part of the sum, and O^T.
template <class C>
struct AttendState {
  float mx[C::NT], ms[C::NT], l[C::NT];
  f32x4 o[C::NT][C::DT];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      mx[nt] = neg_inf();
      ms[nt] = l[nt] = 0.f;
#pragma unroll
      for (int d = 0; d < C::DT; ++d) o[nt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
};

// Raises the reference m of a wave's rows where one of the scores of NX
// 16-key blocks asks for it.
template <class C, int NX>
__device__ __forceinline__ void raise_reference(float c,
                                                const f32x4 (&s)[C::NT][NX],
                                                AttendState<C>& st) {
  bool up = false;
  float tm[C::NT];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    tm[nt] = s[nt][0][0];
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) tm[nt] = fmaxf(tm[nt], s[nt][x][e]);
    tm[nt] *= c;
    up = up || tm[nt] > st.mx[nt] + kRaise;
  }
  if (__ballot(up)) {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      const float m2 = fmaxf(st.mx[nt], row_max(tm[nt]));
      const float f =
          m2 == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(st.mx[nt] - m2);
      st.mx[nt] = m2;
      st.ms[nt] = m2 == neg_inf() ? 0.f : m2 - kLift<C::BF16>;
      st.l[nt] *= f;
#pragma unroll
      for (int d = 0; d < C::DT; ++d) st.o[nt][d] *= f;
    }
  }
}

// Probabilities of 32 keys (the 16-key blocks x0 and x0 + 1 of s), rounded to
// the type of the values they meet, as B operands.
template <class C, int NX>
__device__ __forceinline__ void probabilities(float c,
                                              const f32x4 (&s)[C::NT][NX],
                                              int x0, AttendState<C>& st,
                                              s16x8 (&pf)[C::NT]) {
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    f32x8 p;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p[e] = __builtin_amdgcn_exp2f(
          __builtin_fmaf(s[nt][x0 + e / 4][e & 3], c, -st.ms[nt]));
    st.l[nt] += ((p[0] + p[1]) + (p[2] + p[3])) +
                ((p[4] + p[5]) + (p[6] + p[7]));
    pf[nt] = round8<C::BF16>(p);
  }
}

// Adds the elements of the value at position t that are not finite to the
// rows of block nt that see it (the tile holds 0 in their place); sk: the
// rows' scores, -inf where it is not seen, in the lanes of quad `from`.
template <class C>
__device__ __forceinline__ void add_odd_value(const AttendArgs& a,
                                              const int32_t* table, int h,
                                              int t, int nt, float sk,
                                              int from, AttendState<C>& st) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const PageGeom& g = a.g;
  const int D = opaque(g.D);
  const int p = table[t >> g.shift];
  const uint16_t* v =
      static_cast<const uint16_t*>(a.vc) +
      ((((int64_t)p * g.Hkv + h) << g.shift) + (t & ((1 << g.shift) - 1))) * D;
  sk = __shfl(sk, from * 16 + col, kWave);
  const float pk = __builtin_amdgcn_exp2f(__builtin_fmaf(sk, a.c, -st.ms[nt]));
#pragma unroll
  for (int d = 0; d < C::DT; ++d) {
    if (16 * d >= D) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = elem<C::BF16>(v[16 * d + 4 * quad + e]);
      if (sk != neg_inf() && !(fabsf(x) < pos_inf())) st.o[nt][d][e] += pk * x;
    }
  }
}

// Takes the elements of a 16-byte piece that are not finite out of it;
// returns whether there were any.
template <bool BF16>
__device__ __forceinline__ bool drop_odd(uint4& v) {
  // without its sign an element that is not finite is at least inf's bits:
  // adding what is missing to 0x8000 carries into the sign bit
  constexpr uint32_t inf = BF16 ? 0x7f80u : 0x7c00u;
  constexpr uint32_t add = (0x8000u - inf) * 0x10001u;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t any = ((w[0] & 0x7fff7fffu) + add) |
                       ((w[1] & 0x7fff7fffu) + add) |
                       ((w[2] & 0x7fff7fffu) + add) |
                       ((w[3] & 0x7fff7fffu) + add);
  if (!(any & 0x80008000u)) return false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((w[e] & inf) == inf) w[e] &= 0xffff0000u;
    if ((w[e] & (inf << 16)) == (inf << 16)) w[e] &= 0xffffu;
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  return true;
}

// bits of the keys (lane values) of the lanes with `on`
__device__ __forceinline__ uint64_t key_bits(bool on, int key) {
  uint64_t keys = 0, bal = __ballot(on);
  while (bal) {
    keys |= (uint64_t)1
            << __builtin_amdgcn_readlane(key, __builtin_ctzll(bal));
    bal &= bal - 1;
  }
  return keys;
}

}  // namespace pct
