// k_attend_impl.h -- softmax attention of a round's rows over a paged
// key-value cache, on MFMA.  For a row with the seen positions S,
//   out = sum_{t in S} p_t v_t / sum_{t in S} p_t,  p_t = 2^(z_t - m),
//   z_t = |scale| log2(e) (+-q . k_t),  lse = ln(2) (m + log2 sum p_t),
// in one pass over the positions.  m only has to be near the largest z_t: it
// is raised (and the sums so far are scaled down) when a score comes that
// is more than 2^kRaise above it, so p stays below 2^kRaise and most tiles
// need neither a reduction over lanes nor a rescaling.
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
// group) -> i G + g.  A workgroup of 4 waves works on 16 NT RG of them: RG
// waves share a key tile (16 NT rows each), the KG = 4 / RG key groups take
// different key tiles and join their sums at the end.
//
// Work is the list of all (request, head, row tile, step of KG KB keys),
// cut into equal contiguous runs, one per workgroup, whatever the lengths
// of the requests (known on the device only).  A row tile whose steps lie in
// one run is finished there; otherwise each run leaves its unnormalised
// sums in the workspace and the join kernel adds them up in order of runs,
// so results do not depend on timing.
#pragma once
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr float kRaise = 8.f;

template <int DP_, int NT_, int RG_, int KB_, bool BF16_>
struct AttendCfg {
  static constexpr int DP = DP_;  // head size, padded
  static constexpr int NT = NT_;  // 16-row blocks per wave
  static constexpr int RG = RG_;  // waves that share a key tile
  static constexpr int KB = KB_;  // keys of a tile
  static constexpr bool BF16 = BF16_;
  static constexpr int KG = 4 / RG;
  static constexpr int CH = DP / 8;  // 16-byte pieces of a row
  static constexpr int KS = KB * KG;
  static constexpr int MT = 16 * NT * RG;
  static constexpr int GT = 64 * RG;
  static constexpr int NL = KB * CH / GT;  // pieces of K per thread and tile
  // a wave's own tile needs no second buffer: its LDS operations are in
  // order and the next tile waits in registers
  static constexpr int NBUF = RG == 1 ? 1 : 2;
  // LDS row strides in pieces: odd for K (16 keys of one piece fall on all
  // banks), 2 mod 4 for V (the 32-byte rows of 8 keys that half a
  // transposing read touches fall on all banks)
  static constexpr int KROW = CH + 1, VROW = CH + 2;
  static constexpr int TILE = KB * (KROW + VROW);
  static constexpr int DROW = DP + 4;  // floats of a dumped row of O
  static constexpr int LDS_TILES = KG * NBUF * TILE * 16;
  static constexpr int LDS_DUMP = 4 * 16 * NT * DROW * 4;
  static constexpr int LDS = LDS_TILES > LDS_DUMP ? LDS_TILES : LDS_DUMP;
  static constexpr int OCC = DP <= 128 ? 2 : 1;  // workgroups per CU
  static_assert(KB * CH % GT == 0 && KB % 32 == 0 && KB <= 64, "tile");
};

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

// the lowest n bits (n clamped to [0, 64])
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : (n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1);
}

// Steps of one request.
struct AttendReq {
  int ctx, n, L;  // context, nodes, positions
  int M, RT, KT;  // packed rows, row tiles, steps of a row tile
  int64_t units;  // steps of all heads and row tiles
};
template <int MT, int KS>
__device__ __forceinline__ AttendReq attend_req(const AttendArgs& a, int b) {
  const PageGeom& g = a.g;
  AttendReq r;
  r.n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  r.ctx = clamp_ctx(g.ctx_len[b]);
  r.L = min(r.ctx + r.n + 1, g.max_pages << g.shift);
  r.M = (r.n + 1) * a.G;
  r.RT = (r.M + MT - 1) / MT;
  r.KT = (r.L + KS - 1) / KS;
  r.units = (int64_t)g.Hkv * r.RT * r.KT;
  return r;
}

template <class C>
__global__ __launch_bounds__(256, C::OCC) void attend_kernel(AttendArgs a,
                                                             AttendWs ws) {
  constexpr int NT = C::NT, KB = C::KB, CH = C::CH, NL = C::NL;
  constexpr int KT16 = KB / 16, DT = C::DP / 16, KSTEP = C::DP / 32;
  __shared__ __align__(16) uint4 lds[C::LDS / 16];
  __shared__ int64_t wsum[4];
  __shared__ int64_t seek_off;
  __shared__ int seek_b;
  __shared__ uint64_t flag[C::NBUF][4][2];  // per wave: dead keys, nonfinite
  __shared__ float dump_m[4][16 * NT], dump_l[4][16 * NT];

  const PageGeom& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / C::RG, rg = wave % C::RG;
  const int gtid = tid - kg * C::GT;
  const int col = lane & 15, quad = lane >> 4;

  // ---- this workgroup's run of steps
  const int per = (g.batch + 255) / 256;
  int64_t mine = 0;
  for (int b = tid * per; b < min((tid + 1) * per, g.batch); ++b)
    mine += attend_req<C::MT, C::KS>(a, b).units;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t x = __shfl_up(incl, d, kWave);
    if (lane >= d) incl += x;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) incl += wsum[w];
    total += wsum[w];
  }
  const int n_run = (int)min((int64_t)gridDim.x, total);
  // neighbouring runs on one XCD (workgroups go round the 8 XCDs), so that
  // the row tiles of a head read its keys and values from one L2
  const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
  const int xbase = xcd * (n_run >> 3) + min(xcd, n_run & 7);
  const int xcount = (n_run >> 3) + (xcd < (n_run & 7) ? 1 : 0);
  if (at >= xcount) {
    // runs n_run, ... do not exist: their join entries are empty
    if (tid == 0) {
      int idle = 0;  // idle workgroups before this one
      for (int x = 0; x < 8; ++x) {
        const int c = (n_run >> 3) + (x < (n_run & 7) ? 1 : 0);
        const int have = ((int)gridDim.x - x + 7) >> 3;
        idle += x < xcd ? have - c : 0;
      }
      ws.meta[n_run + idle + at - xcount] = make_int4(0, 0, 0, -1);
    }
    return;
  }
  const int run = xbase + at;
  const int64_t q_run = total / n_run;
  const int r_run = (int)(total - q_run * n_run);
  auto run_start = [&](int w) { return w * q_run + min(w, r_run); };
  int64_t u = run_start(run);
  const int64_t u_end = run_start(run + 1);
  if (incl - mine <= u && u < incl) {
    int64_t off = incl - mine;
    for (int b = tid * per;; ++b) {
      const int64_t n = attend_req<C::MT, C::KS>(a, b).units;
      if (u < off + n) {
        seek_b = b;
        seek_off = off;
        break;
      }
      off += n;
    }
  }
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(seek_b);
  int64_t b_off = seek_off;
  AttendReq rq = attend_req<C::MT, C::KS>(a, b);
  int4 join = make_int4(0, 0, 0, -1);

  const uint4* kc = static_cast<const uint4*>(a.kc);
  const uint4* vc = static_cast<const uint4*>(a.vc);
  const int chd = g.D >> 3;
  const int page_mask = (1 << g.shift) - 1;
  uint4* tiles = lds + kg * C::NBUF * C::TILE;

  while (u < u_end) {
    while (u >= b_off + rq.units) {
      b_off += rq.units;
      rq = attend_req<C::MT, C::KS>(a, ++b);
    }
    const int64_t in = u - b_off;  // step within the request
    const int seg = (int)(in / rq.KT);
    const int k0 = (int)(in - (int64_t)seg * rq.KT);
    const int h = seg / rq.RT, rt = seg - h * rq.RT;
    const int k1 = (int)min((int64_t)rq.KT, k0 + (u_end - u));
    const int ctx = rq.ctx, L = rq.L;
    const int32_t* table = g.table + (int64_t)b * g.max_pages;

    // ---- query rows of this wave
    int irow[NT];
    s16x8 qf[NT][KSTEP];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int m = rt * C::MT + (rg * NT + nt) * 16 + col;
      const int i = m / a.G;
      irow[nt] = i;
      const bool ok = m < rq.M;
      const uint4* q = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.q) +
          ((int64_t)b * (g.N + 1) + (ok ? i : 0)) * a.qs +
          (h * a.G + (ok ? m - i * a.G : 0)) * g.D);
#pragma unroll
      for (int s = 0; s < KSTEP; ++s) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (ok && 4 * s + quad < chd) x = q[4 * s + quad];
        // the sign of the scale; a scale of zero leaves zeros
        x.x = (x.x & a.qand) ^ a.qxor;
        x.y = (x.y & a.qand) ^ a.qxor;
        x.z = (x.z & a.qand) ^ a.qxor;
        x.w = (x.w & a.qand) ^ a.qxor;
        qf[nt][s] = __builtin_bit_cast(s16x8, x);
      }
    }
    f32x4 o[NT][DT];
    float mx[NT], ms[NT], l[NT];  // ms: mx, 0 while nothing was seen
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt] = neg_inf();
      ms[nt] = 0.f;
      l[nt] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[nt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // ---- key tiles: pages two tiles ahead, pieces one tile ahead
    uint4 kr[NL], vr[NL];
    int page[NL];
    uint32_t dead = 0;  // bit j: piece j has no page
    auto tile_t0 = [&](int k) { return k * C::KS + kg * KB; };
    auto key_of = [&](int j) { return (j * C::GT + gtid) / CH; };
    auto piece_of = [&](int j) { return (j * C::GT + gtid) % CH; };
    auto load_pages = [&](int k) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        page[j] = table[min(tile_t0(k) + key_of(j), L - 1) >> g.shift];
    };
    auto load_rows = [&](int k) __attribute__((always_inline)) {
      dead = 0;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int t = min(tile_t0(k) + key_of(j), L - 1);
        int p = page[j];
        if ((unsigned)p >= (unsigned)g.n_pages) {
          p = 0;
          dead |= 1u << j;
        }
        const int64_t row =
            (((int64_t)p * g.Hkv + h) << g.shift) + (t & page_mask);
        const int c = piece_of(j);
        kr[j] = vr[j] = make_uint4(0, 0, 0, 0);
        if (c < chd) {
          kr[j] = kc[row * chd + c];
          vr[j] = vc[row * chd + c];
        }
      }
    };
    load_pages(k0);
    load_rows(k0);
    if (k0 + 1 < k1) load_pages(k0 + 1);

    for (int k = k0; k < k1; ++k) {
      const int buf = C::NBUF == 1 ? 0 : (k - k0) & 1;
      uint4* kt = tiles + buf * C::TILE;
      uint4* vt = kt + KB * C::KROW;
      const int t0 = tile_t0(k);
      const bool tail = t0 + KB > ctx + 1;  // nodes, or past the end

      // ---- the tile from registers to LDS
      uint64_t dead_keys = 0, odd_keys = 0;
      if (tail) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int t = t0 + key_of(j);
          if (t >= L) vr[j] = make_uint4(0, 0, 0, 0);
          // A node's value that is not finite must not meet the
          // probability 0 of a row that does not see it: it is taken out
          // here and added to the rows that see it below.
          bool odd = false;
          uint32_t w[4] = {vr[j].x, vr[j].y, vr[j].z, vr[j].w};
          const uint32_t ex = C::BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((w[e] & ex) == ex) {
              odd = true;
              w[e] &= 0xffff0000u;
            }
            if ((w[e] & (ex << 16)) == (ex << 16)) {
              odd = true;
              w[e] &= 0xffffu;
            }
          }
          odd = odd && t > ctx && !((dead >> j) & 1);
          if (odd) vr[j] = make_uint4(w[0], w[1], w[2], w[3]);
          uint64_t bal = __ballot(odd);
          while (bal) {
            const int src = __builtin_ctzll(bal);
            odd_keys |= (uint64_t)1
                        << __builtin_amdgcn_readlane(key_of(j), src);
            bal &= bal - 1;
          }
        }
      }
      if (__ballot(dead != 0)) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const bool d = (dead >> j) & 1;
          if (d) vr[j] = make_uint4(0, 0, 0, 0);
          uint64_t bal = __ballot(d);
          while (bal) {
            const int src = __builtin_ctzll(bal);
            dead_keys |= (uint64_t)1
                         << __builtin_amdgcn_readlane(key_of(j), src);
            bal &= bal - 1;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        kt[key_of(j) * C::KROW + piece_of(j)] = kr[j];
        vt[key_of(j) * C::VROW + piece_of(j)] = vr[j];
      }
      if (C::RG > 1 && lane == 0) {
        flag[buf][wave][0] = dead_keys;
        flag[buf][wave][1] = odd_keys;
      }
      if (k + 1 < k1) load_rows(k + 1);
      if (k + 2 < k1) load_pages(k + 2);
      if (C::RG > 1) {
        __syncthreads();
#pragma unroll
        for (int w = 0; w < C::RG; ++w) {
          dead_keys |= flag[buf][kg * C::RG + w][0];
          odd_keys |= flag[buf][kg * C::RG + w][1];
        }
      } else {
        __builtin_amdgcn_wave_barrier();
      }

      // ---- scores
      f32x4 s[NT][KT16];
#pragma unroll
      for (int x = 0; x < KT16; ++x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < KSTEP; ++st) {
          const s16x8 kf = __builtin_bit_cast(
              s16x8, kt[(16 * x + col) * C::KROW + 4 * st + quad]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            s[nt][x] = mfma16<C::BF16>(kf, qf[nt][st], s[nt][x]);
        }
      }

      // ---- mask of a tile with nodes, with missing pages or past the end
      const bool edge = tail || dead_keys != 0;
      if (edge) {
        const uint64_t all = low_bits(L - t0) & ~dead_keys;
        const int j0 = t0 - ctx - 1;  // node of the tile's first key
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int i = irow[nt];
          uint64_t see = low_bits(-j0);  // the context and the root
          if (i > 0 && i <= rq.n) {
            if (a.mask == nullptr) {
              see |= low_bits(i - j0);
            } else if (j0 > -64) {
              const uint64_t* mr =
                  a.mask + ((int64_t)b * g.N + i - 1) * a.words;
              if (j0 < 0) {
                see |= mr[0] << -j0;
              } else {
                const int w = j0 >> 6, sh = j0 & 63;
                if (w < a.words) see |= mr[w] >> sh;
                if (sh != 0 && w + 1 < a.words) see |= mr[w + 1] << (64 - sh);
              }
            }
          }
          see = (see & all) >> (4 * quad);
#pragma unroll
          for (int x = 0; x < KT16; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((see >> (16 * x + e)) & 1)) s[nt][x][e] = neg_inf();
        }
      }

      // ---- probabilities
      s16x8 pf[NT][KT16 / 2];
      bool up = false;
      float tm[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        tm[nt] = s[nt][0][0];
#pragma unroll
        for (int x = 0; x < KT16; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) tm[nt] = fmaxf(tm[nt], s[nt][x][e]);
        tm[nt] *= a.c;
        up = up || tm[nt] > mx[nt] + kRaise;
      }
      if (__ballot(up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m2 = fmaxf(mx[nt], row_max(tm[nt]));
          const float f =
              m2 == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(mx[nt] - m2);
          mx[nt] = m2;
          ms[nt] = m2 == neg_inf() ? 0.f : m2;
          l[nt] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[nt][d] *= f;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int y = 0; y < KT16 / 2; ++y) {
          f32x8 p;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(
                s[nt][2 * y + e / 4][e & 3], a.c, -ms[nt]));
            l[nt] += p[e];
          }
          // a probability is rounded to the type of the values it meets
          pf[nt][y] = round8<C::BF16>(p);
        }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int y = 0; y < KT16 / 2; ++y) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const uint16_t* vb = reinterpret_cast<const uint16_t*>(vt) +
                               (32 * y + 4 * quad + (col >> 2)) *
                                   (8 * C::VROW) +
                               16 * d + 4 * (col & 3);
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(const_cast<uint16_t*>(vb)));
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(const_cast<uint16_t*>(vb + 16 * 8 * C::VROW)));
          const s16x8 vf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5,
                                                   6, 7);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            o[nt][d] = mfma16<C::BF16>(vf, pf[nt][y], o[nt][d]);
        }
      }

      // ---- values that are not finite, for the rows that see them
      while (odd_keys) {
        const int key = __builtin_ctzll(odd_keys);
        odd_keys &= odd_keys - 1;
        const int t = t0 + key;
        const int p = table[t >> g.shift];
        const uint16_t* v =
            reinterpret_cast<const uint16_t*>(vc) +
            ((((int64_t)p * g.Hkv + h) << g.shift) + (t & page_mask)) * g.D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float sk = 0.f;
#pragma unroll
          for (int x = 0; x < KT16; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key >> 4 == x && (key & 3) == e) sk = s[nt][x][e];
          sk = __shfl(sk, ((key >> 2) & 3) * 16 + col, kWave);
          const float pk =
              __builtin_amdgcn_exp2f(__builtin_fmaf(sk, a.c, -ms[nt]));
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            if (16 * d >= g.D) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = elem<C::BF16>(v[16 * d + 4 * quad + e]);
              if (sk != neg_inf() && !(fabsf(x) < pos_inf()))
                o[nt][d][e] += pk * x;
            }
          }
        }
      }
    }

    // ---- sums to LDS, joined over the key groups
    __syncthreads();
    float* dump = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ls = row_sum(l[nt]);
      float* to = dump + (wave * 16 * NT + 16 * nt + col) * C::DROW + 4 * quad;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4*>(to + 16 * d) = o[nt][d];
      if (quad == 0) {
        dump_m[wave][16 * nt + col] = mx[nt];
        dump_l[wave][16 * nt + col] = ls;
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == rq.KT;
    const int slot = 2 * run + (k0 == 0 ? 1 : 0);
    float* part_o = ws.o + (int64_t)slot * C::MT * C::DP;
    float2* part_ml = ws.ml + (int64_t)slot * C::MT;
    for (int x = tid; x < C::MT * CH; x += 256) {
      const int r = x / CH, c = x - r * CH;  // row of the tile, piece
      const int m = rt * C::MT + r;
      if (m >= rq.M || c >= chd) continue;
      const int w0 = r / (16 * NT), rr = r - w0 * 16 * NT;
      float top = neg_inf();
#pragma unroll
      for (int y = 0; y < C::KG; ++y)
        top = fmaxf(top, dump_m[y * C::RG + w0][rr]);
      float sum = 0.f;
      f32x8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < C::KG; ++y) {
        const int w = y * C::RG + w0;
        const float f =
            top == neg_inf()
                ? 0.f
                : __builtin_amdgcn_exp2f(dump_m[w][rr] - top);
        sum += f * dump_l[w][rr];
        const f32x4* from = reinterpret_cast<const f32x4*>(
            dump + (w * 16 * NT + rr) * C::DROW + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f * from[e >> 2][e & 3];
      }
      if (whole) {
        const int i = m / a.G;
        const int64_t row = ((int64_t)b * (g.N + 1) + i) * a.Hq + h * a.G +
                            (m - i * a.G);
        // nothing seen: zero (a NaN stays one)
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        static_cast<uint4*>(a.out)[row * chd + c] =
            __builtin_bit_cast(uint4, round8<C::BF16>(acc * inv));
        if (a.lse && c == 0)
          a.lse[row] = sum == 0.f
                           ? neg_inf()
                           : (top + __builtin_log2f(sum)) * (float)kLn2;
      } else {
        *reinterpret_cast<f32x8*>(part_o + r * C::DP + 8 * c) = acc;
        if (c == 0) part_ml[r] = make_float2(top, sum);
      }
    }
    if (!whole && k0 == 0) {
      // the join adds the runs up to the one that holds the last step
      const int64_t last = u + (rq.KT - k0) - 1;
      const int64_t big = (int64_t)r_run * (q_run + 1);
      const int w1 = (int)(last < big ? last / (q_run + 1)
                                      : r_run + (last - big) / q_run);
      join = make_int4(b, h, rt, w1);
    }
    __syncthreads();
    u += k1 - k0;
  }
  if (tid == 0) ws.meta[run] = join;
}

template <class C>
hipError_t launch_attend_cfg(const AttendArgs& a, const AttendWs& ws,
                             int n_wg, hipStream_t s) {
  hipLaunchKernelGGL(attend_kernel<C>, dim3(n_wg), dim3(256), 0, s, a, ws);
  return hipGetLastError();
}

// keys of a tile by head size and waves that share it
constexpr int attend_kb(int DP, int RG) { return RG == 4 && DP < 256 ? 64 : 32; }

template <int DP>
hipError_t launch_attend_dp(const AttendArgs& a, const AttendPlan& p,
                            const AttendWs& ws, hipStream_t s) {
#define PCT_ATTEND(NT, RG)                                                   \
  if (p.nt == NT && p.rg == RG) {                                            \
    if (a.bf16)                                                              \
      return launch_attend_cfg<                                              \
          AttendCfg<DP, NT, RG, attend_kb(DP, RG), true>>(a, ws, p.n_wg, s); \
    return launch_attend_cfg<                                                \
        AttendCfg<DP, NT, RG, attend_kb(DP, RG), false>>(a, ws, p.n_wg, s);  \
  }
  PCT_ATTEND(1, 1)
  PCT_ATTEND(2, 1)
  PCT_ATTEND(2, 2)
  PCT_ATTEND(2, 4)
#undef PCT_ATTEND
  return hipErrorInvalidValue;
}

}  // namespace pct
