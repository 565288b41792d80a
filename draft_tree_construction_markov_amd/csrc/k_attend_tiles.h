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
// s ^ fV(r) of V, so that the 16 keys of an operand read, and the 8 keys of
// half a transposing read, fall on all banks.  Slots past the head size are
// never loaded and stay zero.
#pragma once
#include "k_attend_impl.h"

namespace pct {

typedef __attribute__((address_space(3))) void* lds_any;

template <int DP_, int NT_, bool BF16_>
struct TilesCfg {
  static constexpr int DP = DP_;  // head size, padded
  static constexpr int NT = NT_;  // 16-row blocks per wave
  static constexpr bool BF16 = BF16_;
  static constexpr int SL = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;
  static constexpr int KB = DP <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int DT = DP / 16, KSTEP = DP / 32;
  static constexpr int GD = DT % 4 == 0 ? 4 : 2;  // V operands of a group
  static constexpr int KS = KB;
  static constexpr int MT = 64 * NT;
  static constexpr int RPI = 64 / SL;       // rows per direct load
  static constexpr int NI = KB / 4 / RPI;   // direct loads of K per wave
  static constexpr int GPS = KB / 8;        // 8-key groups of a tile
  static constexpr int TPV = 64 / GPS;      // tiles whose pages fit a wave
  static constexpr int OCC = DP <= 128 ? 2 : 1;  // workgroups per CU
  static __device__ __forceinline__ int swizzle_k(int r) {
    return SL == 8 ? (r >> 1) & 7 : r & 15;
  }
  static __device__ __forceinline__ int swizzle_v(int r) {
    return 2 * (SL == 8 ? (r >> 1) & 3 : r & 7);
  }
};

// 16 bytes per lane from base + off straight to LDS slots to[lane]; base,
// bytes and to are the same in every lane, off + 16 past `bytes` reads
// nothing.
__device__ __forceinline__ void load_to_lds(const uint4* base, int bytes,
                                            int off, uint4* to) {
#if defined(__HIP_DEVICE_COMPILE__)  // the buffer type exists there only
  const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint4*>(base),
                                                   0, bytes, 0x00027000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_any)to, 16, off, 0, 0, 0);
#endif
}

template <class C>
__global__ __launch_bounds__(256, C::OCC) void attend_tiles_kernel(
    AttendArgs a, AttendWs ws) {
  constexpr int NT = C::NT, KB = C::KB, SL = C::SL, NI = C::NI;
  constexpr int DT = C::DT, KSTEP = C::KSTEP, GD = C::GD;
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

  // direct loads: this lane's row of load 0 and its pieces there.  Load i
  // reads rows i RPI further; the bits of a row and of i RPI are distinct, so
  // its swizzle differs by that of i RPI.
  const int row0 = wave * (KB / 4) + lane / SL;
  const int kp0 = (lane % SL) ^ C::swizzle_k(row0);
  const int vp0 = (lane % SL) ^ C::swizzle_v(row0);
  const int row_bytes = chd * 16, group_bytes = 8 * row_bytes;

  // operand reads: bytes of K for the first 32 elements, of V for the first
  // 16; later ones differ in bits of the swizzled slot only
  const int kx = (col * SL + (quad ^ C::swizzle_k(col))) * 16;
  const int vkey = 4 * quad + (col >> 2);
  const int vx = (vkey * SL + C::swizzle_v(vkey)) * 16 + (col & 3) * 8;

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
      if (small) {
        // a page of its own for every row: through registers
#pragma unroll 1
        for (int x = tid; x < KB * SL; x += 256) {
          const int r = x / SL, sl = x % SL;
          const int t = min(k * KB + r, L - 1);
          int p = table[t >> g.shift];
          p = (unsigned)p < (unsigned)g.n_pages ? p : 0;
          const int64_t at =
              ((((int64_t)p * g.Hkv + h) << g.shift) + (t & page_mask)) * chd;
          const int kp = sl ^ C::swizzle_k(r), vp = sl ^ C::swizzle_v(r);
          if (kp < chd) kd[x] = static_cast<const uint4*>(a.kc)[at + kp];
          if (vp < chd) vd[x] = static_cast<const uint4*>(a.vc)[at + vp];
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
      const int lr = opaque((lane / SL) * row_bytes);
      const int kp = opaque(kp0), vp = opaque(vp0);
      // bytes of a piece from its 8-key group on; a slot past the head size
      // gets an offset past the group, which the bound of the buffer
      // descriptor keeps from being read
      auto bytes = [&](int piece, int i) {
        const int off = lr + (i * C::RPI & 7) * row_bytes + piece * 16;
        return piece < chd ? off : group_bytes;
      };
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int grp = (wave * (KB / 4) + i * C::RPI) >> 3;
        int p = __builtin_amdgcn_readlane(pv, first + grp);
        p = (unsigned)p < (unsigned)g.n_pages ? p : 0;
        const int64_t at = ((((int64_t)p * g.Hkv + h) << g.shift) +
                            ((k * KB + 8 * grp) & page_mask)) * chd;
        load_to_lds(static_cast<const uint4*>(a.kc) + at, group_bytes,
                    bytes(kp ^ C::swizzle_k(i * C::RPI), i),
                    kd + (wave * NI + i) * 64);
        load_to_lds(static_cast<const uint4*>(a.vc) + at, group_bytes,
                    bytes(vp ^ C::swizzle_v(i * C::RPI), i),
                    vd + (wave * NI + i) * 64);
      }
      return ((no_page >> first) & low_bits(C::GPS)) != 0;
    };

    // operands of the 16-key block x of the tile in kt, and their products
    auto read_k = [&](const uint4* kt, int x, int kx0, s16x8(&kf)[KSTEP])
        __attribute__((always_inline)) {
      const char* kb =
          reinterpret_cast<const char*>(kt) + 16 * x * SL * 16;
#pragma unroll
      for (int z = 0; z < KSTEP; ++z)
        kf[z] = *reinterpret_cast<const s16x8*>(kb + (kx0 ^ (64 * z)));
    };
    auto scores = [&](const s16x8(&kf)[KSTEP], int nt)
        __attribute__((always_inline)) {
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int z = 0; z < KSTEP; ++z)
        s = mfma16<C::BF16>(kf[z], qf[nt][z], s);
      return s;
    };
    // operands of keys 32 y .. and elements 16 GD d0 .. of the tile in vt, and
    // their products
    auto read_v = [&](const uint4* vt, int y, int d0, int vx0,
                      s16x8(&vf)[GD]) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < GD; ++d) {
        char* vb = const_cast<char*>(reinterpret_cast<const char*>(vt)) +
                   (vx0 ^ (32 * (GD * d0 + d))) + 32 * y * SL * 16;
        const s16x4 lo =
            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)vb);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4)(vb + 16 * SL * 16));
        vf[d] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
    };
    auto values = [&](const s16x8(&vf)[GD], int d0, const s16x8(&pf)[NT])
        __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < GD; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          st.o[nt][GD * d0 + d] =
              mfma16<C::BF16>(vf[d], pf[nt], st.o[nt][GD * d0 + d]);
    };
    // every wave's loads of the current tile have arrived, and every wave is
    // done with the other buffer
    auto arrived = [&]() __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    };

    bool holes = false;  // the next tile has keys without a page
    // a tile of context whose keys all have pages
    auto tile = [&](int k, const uint4* kt, const uint4* vt, uint4* kn,
                    uint4* vn) __attribute__((always_inline)) {
      arrived();
      if (k + 1 < k1) holes = issue(k + 1, kn, vn);
      // Operands are read one group of products ahead; the barriers keep the
      // compiler from moving a group's reads back to its products.
      constexpr int NX = KB / 16, NG = DT / GD, NV = KB / 32 * NG;
      f32x4 s[NT][NX];
      s16x8 kf[2][KSTEP], vf[2][GD], pf[NT];
      const int kx0 = opaque(kx), vx0 = opaque(vx);
      read_k(kt, 0, kx0, kf[0]);
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        if (x + 1 < NX)
          read_k(kt, x + 1, kx0, kf[(x + 1) & 1]);
        else
          read_v(vt, 0, 0, vx0, vf[0]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][x] = scores(kf[x & 1], nt);
        __builtin_amdgcn_sched_barrier(0);
      }
      raise_reference<C, NX>(a.c, s, st);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i % NG == 0) probabilities<C, NX>(a.c, s, 2 * (i / NG), st, pf);
        if (i + 1 < NV)
          read_v(vt, (i + 1) / NG, (i + 1) % NG, vx0, vf[(i + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
        values(vf[i & 1], i % NG, pf);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // any other tile
    auto edge_tile = [&](int k, const uint4* kt, uint4* vt, uint4* kn,
                         uint4* vn) __attribute__((always_inline)) {
      arrived();
      if (k + 1 < k1) holes = issue(k + 1, kn, vn);
      // keys that exist and have a page
      const int t0 = k * KB;
      bool on = lane < KB && t0 + lane < L;
      if (on)
        on = (unsigned)table[(t0 + lane) >> g.shift] < (unsigned)g.n_pages;
      const uint64_t all = __ballot(on);
      // Values of other keys become 0.  A node's value that is not finite
      // must not meet the probability 0 of a row that does not see it: it is
      // taken out here and added to the rows that see it below.
      uint64_t odd_keys = 0;
#pragma unroll 1
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

#pragma unroll 1
      for (int y = 0; y < KB / 32; ++y) {
        f32x4 s[NT][2];
        s16x8 pf[NT];
        uint32_t see[NT];
        const int kx0 = opaque(kx);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s16x8 kf[KSTEP];
          read_k(kt, 2 * y + x, kx0, kf);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][x] = scores(kf, nt);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          see[nt] = (uint32_t)(seen_keys(a, b, irow[nt], rq.n, ctx,
                                         t0 + 32 * y) & (all >> (32 * y)));
        mask_scores<C>(see, s);
        raise_reference<C, 2>(a.c, s, st);
        probabilities<C, 2>(a.c, s, 0, st, pf);
        const int vx0 = opaque(vx);
#pragma unroll
        for (int i = 0; i < DT / GD; ++i) {
          s16x8 vf[GD];
          read_v(vt, y, i, vx0, vf);
          values(vf, i, pf);
        }
        add_odd_values<C>(a, table, h, t0 + 32 * y,
                          (uint32_t)(odd_keys >> (32 * y)), s, st);
      }
    };

    __syncthreads();  // the previous run's last tile has been read
    holes = issue(k0, k_a, v_a);
    // Tiles of context go in pairs through the fast path (its loop names the
    // buffers); an odd one, nodes and holes take the other path.
    auto clean = [&](int k) {
      return k < k1 && !holes && (k + 1) * KB <= ctx + 1;
    };
    for (int k = k0, par = 0; k < k1; ++k, par ^= 1) {
      if (par == 0) {
        while (clean(k)) {
          tile(k, k_a, v_a, k_b, v_b);
          ++k;
          par = 1;
          if (!clean(k)) break;
          tile(k, k_b, v_b, k_a, v_a);
          ++k;
          par = 0;
        }
        if (k >= k1) break;
      }
      edge_tile(k, par ? k_b : k_a, par ? v_b : v_a, par ? k_a : k_b,
                par ? v_a : v_b);
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
