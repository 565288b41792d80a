// k_attend_tiles.h -- attention of more than 32 packed rows per key-value
// head (draft trees, pieces of prompts): the 4 waves of a workgroup hold 16 NT
// rows each and share every key tile.  Tiles go from the cache straight to
// LDS (16-byte direct loads) into two buffers, so the next tile's loads are
// in flight while the current one is multiplied; the two buffers are
// distinct LDS objects and the loop is unrolled by two, which lets the
// compiler see that the reads of one do not wait for the loads of the other.
//
// LDS layout: rows of SL 16-byte slots without padding (direct loads write
// 64 consecutive slots per wave instruction), swizzled by the choice of the
// piece that a lane loads: slot s of key r holds piece s ^ fK(r) of K, and
// s ^ 2 fV(r) of V, so that the 16 keys of an operand read, and the 8 keys of
// half a transposing read, fall on all banks.  Slots past the head size are
// never loaded and stay zero.
#pragma once
#include "k_attend_impl.h"

namespace pct {

typedef __attribute__((address_space(3))) void* lds_any;
typedef const __attribute__((address_space(1))) void* gbl_any;

template <int DP_, int NT_, bool BF16_>
struct TilesCfg {
  static constexpr int DP = DP_;  // head size, padded
  static constexpr int NT = NT_;  // 16-row blocks per wave
  static constexpr bool BF16 = BF16_;
  static constexpr int SL = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;
  static constexpr int KB = DP <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int KT16 = KB / 16, DT = DP / 16, KSTEP = DP / 32;
  static constexpr int KS = KB;
  static constexpr int MT = 64 * NT;
  static constexpr int RPI = 64 / SL;       // rows per direct load
  static constexpr int NI = KB / 4 / RPI;   // direct loads of K per wave
  static constexpr int GPS = KB / 8;        // 8-key groups of a tile
  static constexpr int TPV = 64 / GPS;      // tiles whose pages fit a wave
  static constexpr int OCC = DP <= 128 ? 2 : 1;  // workgroups per CU
};

template <class C>
__global__ __launch_bounds__(256, C::OCC) void attend_tiles_kernel(
    AttendArgs a, AttendWs ws) {
  constexpr int NT = C::NT, KB = C::KB, SL = C::SL, NI = C::NI;
  constexpr int KT16 = C::KT16, DT = C::DT, KSTEP = C::KSTEP;
  __shared__ __align__(16) uint4 k_a[KB * SL];
  __shared__ __align__(16) uint4 v_a[KB * SL];
  __shared__ __align__(16) uint4 k_b[KB * SL];
  __shared__ __align__(16) uint4 v_b[KB * SL];
  __shared__ uint64_t odd_s[4];

  const PageGeom& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;

  AttendRun run;
  if (!attend_schedule<C::MT, C::KS>(a, ws, run)) return;
  int b = run.b;
  int64_t u = run.u, b_off = run.b_off;
  AttendReq rq = attend_req<C::MT, C::KS>(a, b);
  int4 join = make_int4(0, 0, 0, -1);

  const int chd = g.D >> 3;
  const int page_mask = (1 << g.shift) - 1;
  const bool small = g.shift < 3;  // pages end inside the 8-key groups
  if (chd < SL) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < KB * SL; i += 256)
      k_a[i] = v_a[i] = k_b[i] = v_b[i] = zero;
  }

  // direct loads: this lane's row within its 8-key group and its pieces
  const int row0 = wave * (KB / 4) + lane / SL;  // row of load 0 in the tile
  int koff[NI], voff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = row0 + i * C::RPI, s = lane % SL;
    const int fk = SL == 8 ? (r >> 1) & 7 : r & 15;
    const int fv = SL == 8 ? (r >> 1) & 3 : r & 7;
    const int kp = s ^ fk, vp = s ^ (2 * fv);
    koff[i] = kp < chd ? (r & 7) * chd + kp : -1;
    voff[i] = vp < chd ? (r & 7) * chd + vp : -1;
  }
  // operand reads: slots of K per 32 elements, bytes of V per 16
  const int fk = SL == 8 ? (col >> 1) & 7 : col;
  const int vkey = 4 * quad + (col >> 2);
  const int fv = SL == 8 ? (vkey >> 1) & 3 : vkey & 7;
  int kx[KSTEP];
#pragma unroll
  for (int z = 0; z < KSTEP; ++z) kx[z] = col * SL + ((4 * z + quad) ^ fk);
  const int vx = vkey * SL * 16 + fv * 32 + (col & 3) * 8;

  while (u < run.end) {
    while (u >= b_off + rq.units) {
      b_off += rq.units;
      rq = attend_req<C::MT, C::KS>(a, ++b);
    }
    const int64_t in = u - b_off;  // step within the request
    const int seg = (int)(in / rq.KT);
    const int k0 = (int)(in - (int64_t)seg * rq.KT);
    const int h = seg / rq.RT, rt = seg - h * rq.RT;
    const int k1 = (int)min((int64_t)rq.KT, k0 + (run.end - u));
    const int ctx = rq.ctx, L = rq.L;
    const int32_t* table = g.table + (int64_t)b * g.max_pages;
    const int m0 = rt * C::MT + wave * 16 * NT;

    int irow[NT];
    s16x8 qf[NT][KSTEP];
    load_queries<C>(a, b, h, m0, rq.M, irow, qf);
    AttendState<C> st;
    st.clear();

    // Pages of the 8-key groups of TPV tiles, one per lane, and of the TPV
    // tiles after them.
    auto group_pages = [&](int k) {
      const int t = (k + lane / C::GPS) * KB + 8 * (lane % C::GPS);
      return table[min(t, L - 1) >> g.shift];
    };
    int kv = k0;
    int pv = group_pages(k0), pv_next = group_pages(k0 + C::TPV);
    uint64_t no_page = __ballot((unsigned)pv >= (unsigned)g.n_pages);

    // issues the loads of tile k; returns whether a group has no page
    auto issue = [&](int k, uint4* kd, uint4* vd)
        __attribute__((always_inline)) -> bool {
      const uint4* kc = static_cast<const uint4*>(a.kc);
      const uint4* vc = static_cast<const uint4*>(a.vc);
      if (small) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = row0 + i * C::RPI;
          const int t = min(k * KB + r, L - 1);
          int p = table[t >> g.shift];
          p = (unsigned)p < (unsigned)g.n_pages ? p : 0;
          const int64_t at =
              ((((int64_t)p * g.Hkv + h) << g.shift) + (t & page_mask) -
               (r & 7)) * chd;
          uint4* kl = kd + (wave * NI + i) * 64;
          uint4* vl = vd + (wave * NI + i) * 64;
          if (koff[i] >= 0)
            __builtin_amdgcn_global_load_lds((gbl_any)(kc + (at + koff[i])),
                                             (lds_any)kl, 16, 0, 0);
          if (voff[i] >= 0)
            __builtin_amdgcn_global_load_lds((gbl_any)(vc + (at + voff[i])),
                                             (lds_any)vl, 16, 0, 0);
        }
        return true;
      }
      if (k - kv >= C::TPV) {
        kv += C::TPV;
        pv = pv_next;
        no_page = __ballot((unsigned)pv >= (unsigned)g.n_pages);
        pv_next = group_pages(kv + C::TPV);
      }
      const int first = (k - kv) * C::GPS;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int grp = (wave * (KB / 4) + i * C::RPI) >> 3;
        int p = __builtin_amdgcn_readlane(pv, first + grp);
        p = (unsigned)p < (unsigned)g.n_pages ? p : 0;
        const int64_t at = ((((int64_t)p * g.Hkv + h) << g.shift) +
                            ((k * KB + 8 * grp) & page_mask)) * chd;
        uint4* kl = kd + (wave * NI + i) * 64;
        uint4* vl = vd + (wave * NI + i) * 64;
        if (koff[i] >= 0)
          __builtin_amdgcn_global_load_lds((gbl_any)(kc + at + koff[i]),
                                           (lds_any)kl, 16, 0, 0);
        if (voff[i] >= 0)
          __builtin_amdgcn_global_load_lds((gbl_any)(vc + at + voff[i]),
                                           (lds_any)vl, 16, 0, 0);
      }
      return ((no_page >> first) & low_bits(C::GPS)) != 0;
    };

    // one tile: wait for its loads, start the next tile's, multiply
    auto tile = [&](int k, const uint4* kt, uint4* vt, uint4* kn, uint4* vn,
                    bool& holes) __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      const int t0 = k * KB;
      const bool edge = holes || t0 + KB > ctx + 1;
      if (k + 1 < k1) holes = issue(k + 1, kn, vn);

      uint64_t odd_keys = 0, all = 0;
      if (edge) {
        // keys that exist and have a page
        const int t = t0 + lane;
        bool on = lane < KB && t < L;
        if (on) on = (unsigned)table[t >> g.shift] < (unsigned)g.n_pages;
        all = __ballot(on);
        // Values of other keys become 0.  A node's value that is not finite
        // must not meet the probability 0 of a row that does not see it:
        // it is taken out here and added to the rows that see it below.
        for (int x = tid; x < KB * SL; x += 256) {
          const int r = x / SL;
          const bool live = (all >> r) & 1;
          uint4 v = vt[x];
          if (!live) vt[x] = make_uint4(0, 0, 0, 0);
          const bool odd = live && t0 + r > ctx && drop_odd<C::BF16>(v);
          if (odd) vt[x] = v;
          odd_keys |= key_bits(odd, r);
        }
        if (lane == 0) odd_s[wave] = odd_keys;
        __syncthreads();
        odd_keys = odd_s[0] | odd_s[1] | odd_s[2] | odd_s[3];
      }

      f32x4 s[NT][KT16];
#pragma unroll
      for (int x = 0; x < KT16; ++x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int z = 0; z < KSTEP; ++z) {
          const s16x8 kf = __builtin_bit_cast(s16x8, kt[16 * SL * x + kx[z]]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            s[nt][x] = mfma16<C::BF16>(kf, qf[nt][z], s[nt][x]);
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t see =
              (seen_keys(a, b, irow[nt], rq.n, ctx, t0) & all) >> (4 * quad);
#pragma unroll
          for (int x = 0; x < KT16; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((see >> (16 * x + e)) & 1)) s[nt][x][e] = neg_inf();
        }
      }
      s16x8 pf[NT][KT16 / 2];
      probabilities<C>(a.c, s, st, pf);
#pragma unroll
      for (int y = 0; y < KT16 / 2; ++y) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          char* vb = reinterpret_cast<char*>(vt) + (vx ^ (32 * d)) +
                     32 * y * SL * 16;
          const s16x4 lo =
              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)vb);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4)(vb + 16 * SL * 16));
          const s16x8 vf =
              __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            st.o[nt][d] = mfma16<C::BF16>(vf, pf[nt][y], st.o[nt][d]);
        }
      }
      if (edge) add_odd_values<C>(a, table, h, t0, odd_keys, s, st);
    };

    __syncthreads();  // the previous run's last tile has been read
    bool holes = issue(k0, k_a, v_a);
    for (int k = k0;;) {
      tile(k, k_a, v_a, k_b, v_b, holes);
      if (++k >= k1) break;
      tile(k, k_b, v_b, k_a, v_a, holes);
      if (++k >= k1) break;
    }

    // ---- finished rows, or sums for the join
    const bool whole = k0 == 0 && k1 == rq.KT;
    const int slot = 2 * run.run + (k0 == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float sum = row_sum(st.l[nt]);
      const int m = m0 + 16 * nt + col;
      if (m >= rq.M) continue;
      if (whole) {
        const int i = irow[nt];
        const int64_t row = ((int64_t)b * (g.N + 1) + i) * a.Hq + h * a.G +
                            (m - i * a.G);
        // nothing seen: zero (a NaN stays one)
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t* to = static_cast<uint16_t*>(a.out) + row * g.D + 4 * quad;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if (16 * d >= g.D) continue;
          *reinterpret_cast<uint2*>(to + 16 * d) =
              round4<C::BF16>(st.o[nt][d] * inv);
        }
        if (a.lse && quad == 0)
          a.lse[row] = sum == 0.f ? neg_inf()
                                  : (st.mx[nt] + __builtin_log2f(sum)) *
                                        (float)kLn2;
      } else {
        const int64_t row =
            (int64_t)slot * C::MT + (wave * NT + nt) * 16 + col;
        float* to = ws.o + row * C::DP + 4 * quad;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<f32x4*>(to + 16 * d) = st.o[nt][d];
        if (quad == 0) ws.ml[row] = make_float2(st.mx[nt], sum);
      }
    }
    if (!whole && k0 == 0) {
      // the join adds the runs up to the one that holds the last step
      join = make_int4(b, h, rt, run.owner(u + rq.KT - 1));
    }
    u += k1 - k0;
  }
  if (tid == 0) ws.meta[run.run] = join;
}

}  // namespace pct
