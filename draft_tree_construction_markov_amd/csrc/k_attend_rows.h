// k_attend_rows.h -- attention of at most 16 packed rows per key-value head
// (plain decoding, short chains): each of a workgroup's 4 waves holds all rows
// and takes its own key tiles, so nothing in the loop waits for another wave;
// the four sums are joined through LDS at the end of a run.  Bound by the
// cache's read: a tile's 16-byte pieces are loaded into registers one tile
// ahead (its pages two ahead) and past the caches (nothing reads them again),
// written to the wave's LDS region and read back as operands.  32 rows per
// wave left no registers for the tile ahead (3.9 TB/s).  Measured with the
// join: 64 requests of one token over up to 32 k positions (2.0 GB) 321 us,
// 6.3 TB/s; one over 131 k positions (0.54 GB) 89 us, 6.0 TB/s (loads that do
// nothing else reach 7.1 on either).  Over 700 positions 10 us, none of it
// bandwidth: schedule 3.6 us with the launch, one tile 4, join 2.3.
#pragma once
#include "k_attend_impl.h"

namespace pct {

template <int DP_, bool BF16_>
struct RowsCfg {
  static constexpr int DP = DP_;  // head size, padded
  static constexpr int NT = 1;     // 16-row blocks
  static constexpr bool BF16 = BF16_;
  static constexpr int KB = kRowsKb;  // keys of a wave's tile
  static constexpr int DT = DP / 16, KSTEP = DP / 32;
  static constexpr int CH = DP / 8;  // 16-byte pieces of a row
  static constexpr int KS = 4 * KB;
  static constexpr int MT = 16 * NT;
  static constexpr int NL = KB * CH / 64;  // pieces of K per lane and tile
  // LDS row strides in pieces: odd for K (16 keys of one piece fall on all
  // banks), 2 mod 4 for V (the 32-byte rows of 8 keys that half a
  // transposing read touches fall on all banks).  One buffer is enough: a
  // wave's LDS operations are in order and the next tile is in registers.
  static constexpr int KROW = CH + 1, VROW = CH + 2;
  static constexpr int TILE = KB * (KROW + VROW);
  static constexpr int DROW = DP + 4;  // floats of a dumped row of O
  static constexpr int LDS_TILES = 4 * TILE * 16;
  static constexpr int LDS_DUMP = 4 * MT * DROW * 4;
  static constexpr int LDS = LDS_TILES > LDS_DUMP ? LDS_TILES : LDS_DUMP;
  static constexpr int OCC = DP <= 128 ? 2 : 1;  // workgroups per CU
  static constexpr int FEW = kRowsFew, LEAST = kRowsLeast;  // of a run
};

// 16 bytes that nothing reads again soon
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(x[0], x[1], x[2], x[3]);
}

template <class C>
__global__ __launch_bounds__(256, C::OCC) void attend_rows_kernel(
    AttendArgs a, AttendWs ws) {
  constexpr int NT = C::NT, KB = C::KB, CH = C::CH, NL = C::NL;
  constexpr int DT = C::DT, KSTEP = C::KSTEP;
  __shared__ __align__(16) uint4 lds[C::LDS / 16];
  __shared__ float dump_m[4][C::MT], dump_l[4][C::MT];

  const PageGeom& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;

  AttendRun run;
  AttendReq rq;
  if (!attend_schedule<C::MT, C::KS, C::FEW, C::LEAST>(a, ws, run, rq)) return;
  i32x4 join = {0, 0, 0, -1};

  const uint4* kc = static_cast<const uint4*>(a.kc);
  const uint4* vc = static_cast<const uint4*>(a.vc);
  const int chd = g.D >> 3;
  const int page_mask = (1 << g.shift) - 1;
  uint4* kt = lds + wave * C::TILE;
  uint4* vt = kt + KB * C::KROW;

  while (run.u < run.end) {
    next_request<C::MT, C::KS>(a, run, rq);
    const int b = run.b;
    const AttendPiece pc = attend_piece(rq, run);
    const int h = pc.h, rt = pc.rt, k0 = pc.k0, k1 = pc.k1;
    const int ctx = rq.ctx, L = rq.L;
    const int32_t* table = g.table + (int64_t)b * g.max_pages;

    int irow[NT];
    s16x8 qf[NT][KSTEP];
    AttendState<C> st;
    st.clear();

    // ---- key tiles: pages two tiles ahead, pieces one tile ahead
    uint4 kr[NL], vr[NL];
    int page[NL];
    uint32_t dead = 0;  // bit j: piece j has no page
    auto tile_t0 = [&](int k) { return k * C::KS + wave * KB; };
    auto key_of = [&](int j) { return (j * 64 + lane) / CH; };
    auto piece_of = [&](int j) { return (j * 64 + lane) % CH; };
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
          kr[j] = load_once(kc + row * chd + c);
          vr[j] = load_once(vc + row * chd + c);
        }
      }
    };
    load_pages(k0);
    load_queries<C>(a, b, h, rt * C::MT, rq.M, irow, qf);
    load_rows(k0);
    if (k0 + 1 < k1) load_pages(k0 + 1);
    note_piece(a, ws, run, rq, pc, join);  // (while these are on their way)
    sign_queries<C>(a, qf);

    for (int k = k0; k < k1; ++k) {
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
          const bool node = t > ctx && t < L && !((dead >> j) & 1);
          odd_keys |= key_bits(node && drop_odd<C::BF16>(vr[j]), key_of(j));
        }
      }
      if (__ballot(dead != 0)) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const bool d = (dead >> j) & 1;
          if (d) vr[j] = make_uint4(0, 0, 0, 0);
          dead_keys |= key_bits(d, key_of(j));
        }
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        kt[key_of(j) * C::KROW + piece_of(j)] = kr[j];
        vt[key_of(j) * C::VROW + piece_of(j)] = vr[j];
      }
      if (k + 1 < k1) load_rows(k + 1);
      if (k + 2 < k1) load_pages(k + 2);
      __builtin_amdgcn_wave_barrier();

      // ---- scores
      f32x4 s[NT][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int z = 0; z < KSTEP; ++z) {
          const s16x8 kf = __builtin_bit_cast(
              s16x8, kt[(16 * x + col) * C::KROW + 4 * z + quad]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            s[nt][x] = mfma16<C::BF16>(kf, qf[nt][z], s[nt][x]);
        }
      }
      // a tile with nodes, with missing pages or past the end
      if (tail || dead_keys != 0) {
        const uint64_t all = low_bits(L - t0) & ~dead_keys;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t see =
              (seen_keys(a, b, irow[nt], rq.n, ctx, t0) & all) >> (4 * quad);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((see >> (16 * x + e)) & 1)) s[nt][x][e] = neg_inf();
        }
      }
      s16x8 pf[NT];
      raise_reference<C, 2>(a.c, s, st);
      probabilities<C, 2>(a.c, s, 0, st, pf);

      // ---- O^T += V^T P^T
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint16_t* vb = reinterpret_cast<const uint16_t*>(vt) +
                             (4 * quad + (col >> 2)) * (8 * C::VROW) + 16 * d +
                             4 * (col & 3);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4)(const_cast<uint16_t*>(vb)));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4)(const_cast<uint16_t*>(vb + 16 * 8 * C::VROW)));
        const s16x8 vf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6,
                                                 7);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          st.o[nt][d] = mfma16<C::BF16>(vf, pf[nt], st.o[nt][d]);
      }
      while (odd_keys) {
        const int key = __builtin_ctzll(odd_keys);
        odd_keys &= odd_keys - 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float sk = 0.f;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key >> 4 == x && (key & 3) == e) sk = s[nt][x][e];
          add_odd_value<C>(a, table, h, t0 + key, nt, sk, (key >> 2) & 3, st);
        }
      }
    }

    // ---- sums to LDS, joined over the waves
    __syncthreads();
    float* dump = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ls = row_sum(st.l[nt]);
      float* to = dump + (wave * C::MT + 16 * nt + col) * C::DROW + 4 * quad;
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<f32x4*>(to + 16 * d) = st.o[nt][d];
      if (quad == 0) {
        dump_m[wave][16 * nt + col] = st.mx[nt];
        dump_l[wave][16 * nt + col] = ls;
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == rq.KT;
    const int slot = 2 * run.run + (k0 == 0 ? 1 : 0);
    float* part_o = ws.o + (int64_t)slot * C::MT * C::DP;
    float2* part_ml = ws.ml + (int64_t)slot * C::MT;
    for (int x = tid; x < C::MT * CH; x += 256) {
      const int r = x / CH, c = x - r * CH;  // row of the tile, piece
      const int m = rt * C::MT + r;
      if (m >= rq.M || c >= chd) continue;
      float top = neg_inf();
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, dump_m[w][r]);
      float sum = 0.f;
      f32x8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = top == neg_inf()
                            ? 0.f
                            : __builtin_amdgcn_exp2f(dump_m[w][r] - top);
        sum += f * dump_l[w][r];
        const f32x4* from = reinterpret_cast<const f32x4*>(
            dump + (w * C::MT + r) * C::DROW + 8 * c);
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
                           : (top + (__builtin_log2f(sum) -
                                     kLift<C::BF16>)) * (float)kLn2;
      } else {
        *reinterpret_cast<f32x8*>(part_o + r * C::DP + 8 * c) = acc;
        if (c == 0) part_ml[r] = make_float2(top, sum);
      }
    }
    __syncthreads();
    run.u += pc.k1 - pc.k0;
  }
  if (tid == 0 && ws.row_tiles == 0) store_meta(ws, run.run, join);
}

}  // namespace pct
