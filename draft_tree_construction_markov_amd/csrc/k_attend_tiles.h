// k_attend_tiles.h -- attention of more than 16 packed rows per key-value
// head (draft trees, pieces of prompts): the W waves of a workgroup hold 16
// NT rows each and share every key tile.  Tiles go from the cache straight to
// LDS (16-byte direct loads) into two buffers, so the next tile's loads are
// in flight while the current one is multiplied.
//
// LDS layout: rows of SL 16-byte slots without padding (direct loads write
// 64 consecutive slots per wave instruction), swizzled by the choice of the
// piece that a lane loads: slot s of key r holds piece s ^ fK(r) of K, and
// s ^ fV(r) of V, so that the 16 keys of an operand read, and the 8 keys of
// half a transposing read, fall on all banks.  Slots past the head size are
// never loaded and stay zero.
//
// Measured, D = 128, 4 query heads per key-value head, with the join: 8
// requests of 256 rows over 33 k positions 1144 us, 968 TFLOP/s (a library's
// 8192^3 product reaches 1160); 32 trees of 257 rows over 512 .. 8192
// positions 633 us, 591 TFLOP/s of work that counts: the ninth row tile of a
// head has 4 rows, and a tile with nodes takes almost twice the 2.3 us of one
// without (masks, the search for values that are not finite).  A step of a
// wave is a chain of products, exponentials and products that two waves per
// SIMD overlap in part; leaving out any one of them (loads, exponentials, the
// second product) saves 4 to 15%, so none of them alone bounds the kernel.
// What did not help: operands read two groups ahead and a check for
// non-finite sums at the end of a piece in place of the search (registers
// spill, and a spill's load waits for the tile under way: +2 .. 4%);
// probabilities before the check of the reference; exponentials between the
// products of the same wave (D = 128 -1%, D = 64 +5%); four blocks of rows
// per wave and one wave per SIMD (half the LDS reads, +45% at D = 64); three
// workgroups per CU at D = 64 (-5 .. +15%).
#pragma once
#include <type_traits>

#include "k_attend_impl.h"

namespace pct {

template <int DP_, int MT_, bool BF16_>
struct TilesCfg {
  static constexpr int DP = DP_;  // head size, padded
  static constexpr int MT = MT_;  // rows of the workgroup: 64 or 128
  // Waves, and 16-row blocks of each: two per operand read from LDS, and two
  // waves per SIMD, as long as the registers hold the sums.  (Wide heads: 16
  // requests of 256 rows over 4352 positions, D = 256, 1130 us with 4 waves
  // of two blocks, one per SIMD, 865 (later 814) with 8 waves of one; D = 192,
  // 829, 685.)
  static constexpr int W = DP > 128 && MT > 64 ? 8 : 4, NT = MT / 16 / W;
  static constexpr bool BF16 = BF16_;
  static constexpr int SL = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;
  static constexpr int KB = kTilesKb;  // keys of a tile
  static constexpr int DT = DP / 16, KSTEP = DP / 32;
  static constexpr int GD = DT % 4 == 0 ? 4 : 2;  // V operands of a group
  static constexpr int KS = KB;
  static constexpr int RPI = 64 / SL;       // rows per direct load
  static constexpr int NI = KB / W / RPI;   // direct loads of K per wave
  static constexpr int GPS = KB / 8;        // 8-key groups of a tile
  static constexpr int TPV = 64 / GPS;      // tiles whose pages fit a wave
  static constexpr int OCC = DP <= 128 ? 2 : 1;  // workgroups per CU
  static constexpr int FEW = kTilesFew, LEAST = tiles_least(MT);  // of a run
  static __device__ __forceinline__ int swizzle_k(int r) {
    return SL == 8 ? (r >> 1) & 7 : r & 15;
  }
  static __device__ __forceinline__ int swizzle_v(int r) {
    return 2 * (SL == 8 ? (r >> 1) & 3 : r & 7);
  }
};

// 16 bytes per lane from base + off straight to the 64 LDS slots at byte
// `to`; base, bytes and to are the same in every lane, off + 16 past `bytes`
// reads nothing.  It is written in assembly because the compiler would
// otherwise wait for the loads of the next tile before every read of the
// current one (both lie in one array): nothing is written to a register,
// and the loop waits for the loads itself, before the barrier that precedes
// the reads.
__device__ __forceinline__ void load_to_lds(const char* base, int bytes,
                                            int off, int to) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const i32x4 rsrc = {
      __builtin_amdgcn_readfirstlane((int)(uint32_t)at),
      __builtin_amdgcn_readfirstlane((int)((at >> 32) & 0xffff)),
      __builtin_amdgcn_readfirstlane(bytes), 0x00027000};
  to = __builtin_amdgcn_readfirstlane(to);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
      "v"(off), "s"(rsrc)
      : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

// The steps [k0, k1) of one row tile, whose rows begin at m0.  Writes finished
// rows, or sums to slot `slot` (of MT rows) for the join.
template <class C>
__device__ __forceinline__ void tiles_piece(
    const AttendArgs& a, const AttendWs& ws, const AttendReq& rq, int b,
    int h, int m0, int k0, int k1, int slot, uint4* tiles,
    uint64_t (*odd_s)[C::W]) {
  constexpr int NT = C::NT, KB = C::KB, SL = C::SL, NI = C::NI, W = C::W;
  constexpr int DT = C::DT, KSTEP = C::KSTEP, GD = C::GD;
  const PageGeom& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int chd = g.D >> 3;
  const int page_mask = (1 << g.shift) - 1;
  const bool small = g.shift < 3;  // pages end inside the 8-key groups
  const int ctx = rq.ctx, L = rq.L;
  const int32_t* table = g.table + (int64_t)b * g.max_pages;

  // direct loads: this lane's row of load 0 and its pieces there.  Load i
  // reads rows i RPI further; the bits of a row and of i RPI are distinct, so
  // its swizzle differs by that of i RPI.
  const int row0 = wave * (KB / W) + lane / SL;
  const int kp0 = (lane % SL) ^ C::swizzle_k(row0);
  const int vp0 = (lane % SL) ^ C::swizzle_v(row0);
  const int row_bytes = chd * 16, group_bytes = 8 * row_bytes;
  // Load i's bytes from the beginning of its 8-key group on; a slot past the
  // head size gets an offset past the group, which the bound of the buffer
  // descriptor keeps from being read.
  int koff[NI], voff[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int off = (lane / SL + (i * C::RPI & 7)) * row_bytes;
    const int kp = kp0 ^ C::swizzle_k(i * C::RPI);
    const int vp = vp0 ^ C::swizzle_v(i * C::RPI);
    koff[i] = kp < chd ? off + kp * 16 : group_bytes;
    voff[i] = vp < chd ? off + vp * 16 : group_bytes;
  }
  // bytes of a page, and of head h within it
  const uint32_t page_bytes = (uint32_t)(g.Hkv * row_bytes) << g.shift;
  const uint32_t head_bytes = (uint32_t)(h * row_bytes) << g.shift;
  const char* k_head = static_cast<const char*>(a.kc) + head_bytes;
  const char* v_head = static_cast<const char*>(a.vc) + head_bytes;
  const int lds0 = __builtin_amdgcn_readfirstlane(
      (int)(uintptr_t)(lds_s16x4)reinterpret_cast<s16x4*>(tiles));
  // operand reads: bytes of K for the first 32 elements, of V for the first
  // 16; later ones differ in bits of the swizzled slot only
  const int kx = (col * SL + (quad ^ C::swizzle_k(col))) * 16;
  const int vkey = 4 * quad + (col >> 2);
  const int vx = (vkey * SL + C::swizzle_v(vkey)) * 16 + (col & 3) * 8;

  // Pages of the 8-key groups of TPV tiles, one per lane, and of the TPV
  // tiles after them.
  auto group_pages = [&](int k) {
    const int t = (k + lane / C::GPS) * KB + 8 * (lane % C::GPS);
    return table[min(t, L - 1) >> g.shift];
  };
  int kv = k0;
  int pv = group_pages(k0), pv_next = group_pages(k0 + C::TPV);

  m0 += 16 * NT * wave;
  const bool idle = m0 >= rq.M;  // a wave without rows loads keys only
  int irow[NT];
  s16x8 qf[NT][KSTEP];
  load_queries<C>(a, b, h, m0, rq.M, irow, qf);
  uint64_t no_page = __ballot((unsigned)pv >= (unsigned)g.n_pages);
  AttendState<C> st;
  st.clear();

  // Mask words of a tile's nodes, loaded with the tile: lane l has the word
  // of the first node for row l % 32 (l % 16 with one block) of the wave's
  // rows if l < 32, else the word after it.
  const int mrow = m0 + (lane & (16 * NT - 1));
  const int node = mrow < rq.M ? mrow / a.G : 0;  // 0: the root
  uint64_t word = 0;
  auto load_word = [&](int k) __attribute__((always_inline)) {
    if (a.mask == nullptr || (k + 1) * KB <= ctx + 1) return;
    const int w = (max(k * KB - ctx - 1, 0) >> 6) + (lane >> 5);
    word = 0;
    if (node > 0 && w < a.words)
      word = a.mask[((int64_t)b * g.N + node - 1) * a.words + w];
  };
  // The keys t0 .. t0 + 63 that the lane's row of block nt sees, as bits
  // (pages and the end of the positions aside).
  auto seen = [&](int nt, int t0) __attribute__((always_inline)) {
    const int j0 = t0 - ctx - 1;   // node of the first key
    uint64_t see = low_bits(-j0);  // the context and the root
    if (a.mask == nullptr) return see | low_bits(irow[nt] - j0);
    const uint64_t lo = shfl_bits(word, 16 * nt + col);
    const uint64_t hi = shfl_bits(word, 32 + 16 * nt + col);
    if (j0 < 0) return j0 > -64 ? see | lo << -j0 : see;
    const int sh = j0 & 63;
    return lo >> sh | (sh != 0 ? hi << (64 - sh) : 0);
  };

  // LDS slots of K of buffer par, followed by those of V
  constexpr int BUF = 2 * KB * SL;
  // issues the loads of this wave's rows of tile k into buffer par; returns
  // whether a group of the tile has no page
  auto issue = [&](int k, int par) __attribute__((always_inline)) -> bool {
    uint4* kd = tiles + par * BUF;
    uint4* vd = kd + KB * SL;
    if (small) {
      // a page of its own for every row: through registers
#pragma unroll 1
      for (int x = wave * (KB / W) * SL + lane; x < (wave + 1) * (KB / W) * SL;
           x += 64) {
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
    int to = lds0 + (par * BUF + wave * NI * 64) * 16;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int grp = (wave * (KB / W) + i * C::RPI) >> 3;
      uint32_t p = __builtin_amdgcn_readlane(pv, first + grp);
      p = p < (uint32_t)g.n_pages ? p : 0;
      const uint64_t at =
          (uint64_t)p * page_bytes +
          (uint32_t)(((k * KB + 8 * grp) & page_mask) * row_bytes);
      load_to_lds(k_head + at, group_bytes, koff[i], to);
      load_to_lds(v_head + at, group_bytes, voff[i], to + KB * SL * 16);
      to += 64 * 16;
    }
    return ((no_page >> first) & low_bits(C::GPS)) != 0;
  };

  // operands of the 16-key block x of the tile in kt, and their products
  auto read_k = [&](const uint4* kt, int x, int kx0, s16x8(&kf)[KSTEP])
      __attribute__((always_inline)) {
    const char* kb = reinterpret_cast<const char*>(kt) + 16 * x * SL * 16;
#pragma unroll
    for (int z = 0; z < KSTEP; ++z)
      kf[z] = *reinterpret_cast<const s16x8*>(kb + (kx0 ^ (64 * z)));
  };
  auto scores = [&](const s16x8(&kf)[KSTEP], f32x4(&s)[NT])
      __attribute__((always_inline)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int z = 0; z < KSTEP; ++z)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        s[nt] = mfma16<C::BF16>(kf[z], qf[nt][z], s[nt]);
  };
  // operands of keys 32 y .. and elements 16 GD d0 .. of the tile in vt, and
  // their products
  auto read_v = [&](const uint4* vt, int y, int d0, int vx0, s16x8(&vf)[GD])
      __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < GD; ++d) {
      char* vb = const_cast<char*>(reinterpret_cast<const char*>(vt)) +
                 (vx0 ^ (32 * (GD * d0 + d))) + 32 * y * SL * 16;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)vb);
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

  bool holes = false;  // the next tile has keys without a page
  // One tile from buffer par, with the loads of the next one into the other
  // under way.  EDGE: a tile with nodes, holes or the end of the positions; other
  // tiles are context that every row sees.
  auto tile = [&](auto edge_c, int k, int par)
      __attribute__((always_inline)) {
    par = __builtin_amdgcn_readfirstlane(par);
    k = __builtin_amdgcn_readfirstlane(k);
    uint4* kt = tiles + par * BUF;
    uint4* vt = kt + KB * SL;
    constexpr bool EDGE = decltype(edge_c)::value;
    constexpr int NX = KB / 16, NG = DT / GD, NV = KB / 32 * NG;
    const int t0 = k * KB;
    uint64_t all = 0, see[NT], odd_keys = 0;
    if constexpr (EDGE) {
      all = low_bits(L - t0);
      if (holes) {
        bool on = lane < KB && t0 + lane < L;
        if (on)
          on = (unsigned)table[(t0 + lane) >> g.shift] < (unsigned)g.n_pages;
        all = __ballot(on);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (EDGE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        see[nt] = (seen(nt, t0) & all) >> (4 * quad);
      // Each wave looks through the values it loaded: those of keys that do
      // not exist become 0.  A node's value that is not finite must not meet
      // the probability 0 of a row that does not see it: it is taken out
      // here and added to the rows that see it below.
      uint4 v[NI];
      const int x0 = wave * (KB / W) * SL + lane;
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = vt[x0 + 64 * i];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = (x0 + 64 * i) / SL;
        const bool live = (all >> r) & 1;
        if (!live) vt[x0 + 64 * i] = make_uint4(0, 0, 0, 0);
        const bool odd = live && t0 + r > ctx && drop_odd<C::BF16>(v[i]);
        if (odd) vt[x0 + 64 * i] = v[i];
        odd_keys |= key_bits(odd, r);
      }
      if (lane == 0) odd_s[par][wave] = odd_keys;
    }
    // every wave's loads of this tile have arrived, and every wave is done
    // with the other buffer
    __syncthreads();
    if (k + 1 < k1) {
      load_word(k + 1);
      holes = issue(k + 1, par ^ 1);
    }
    if (idle) return;
    // Operands are read one group of products ahead; the barriers keep the
    // compiler from moving a group's reads back to its products.
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
      f32x4 sx[NT];
      scores(kf[x & 1], sx);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][x] = sx[nt];
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (EDGE) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((see[nt] >> (16 * x + e)) & 1)) s[nt][x][e] = neg_inf();
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
    if constexpr (EDGE) {
      odd_keys = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) odd_keys |= odd_s[par][w];
      // the scores of these keys once more: it is rare, and they would
      // occupy registers through every tile
      while (odd_keys) {
        const int key = __builtin_ctzll(odd_keys);
        odd_keys &= odd_keys - 1;
        f32x4 sx[NT];
        read_k(kt, key >> 4, kx0, kf[0]);
        scores(kf[0], sx);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int e = key & 3;
          const float se = e == 0   ? sx[nt][0]
                           : e == 1 ? sx[nt][1]
                           : e == 2 ? sx[nt][2]
                                    : sx[nt][3];
          const bool on = (see[nt] >> ((key & ~15) + e)) & 1;
          add_odd_value<C>(a, table, h, t0 + key, nt,
                           on ? se : neg_inf(), (key >> 2) & 3, st);
        }
      }
    }
  };

  __syncthreads();  // the previous piece's last tile has been read
  load_word(k0);
  holes = issue(k0, 0);
  // (the queries' own loads are on their way as well)
  sign_queries<C>(a, qf);
  constexpr std::false_type plain{};
  constexpr std::true_type edge{};
  for (int k = k0, par = 0; k < k1;) {
    // tiles of context that every row sees, in a loop of their own
    while (k < k1 && !holes && (k + 1) * KB <= ctx + 1) {
      tile(plain, k, par);
      ++k;
      par ^= 1;
    }
    if (k >= k1) break;
    tile(edge, k, par);
    ++k;
    par ^= 1;
  }

  // ---- finished rows, or sums for the join
  const bool whole = k0 == 0 && k1 == rq.KT;
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
                                : (st.mx[nt] + (__builtin_log2f(sum) -
                                                kLift<C::BF16>)) *
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
}

template <class C>
__global__ __launch_bounds__(64 * C::W, C::OCC) void attend_tiles_kernel(
    AttendArgs a, AttendWs ws) {
  constexpr int KB = C::KB, SL = C::SL, MT = C::MT;
  __shared__ __align__(16) uint4 tiles[4 * KB * SL];
  __shared__ uint64_t odd_s[2][C::W];

  AttendRun run;
  AttendReq rq;
  if (!attend_schedule<MT, KB, C::FEW, C::LEAST>(a, ws, run, rq)) return;
  i32x4 join = {0, 0, 0, -1};
  if ((a.g.D >> 3) < SL) {
    // slots past the head size are read and never loaded
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < 4 * KB * SL; i += 64 * C::W)
      tiles[i] = zero;
  }
  while (run.u < run.end) {
    next_request<MT, KB>(a, run, rq);
    const int b = run.b;
    const AttendPiece pc = attend_piece(rq, run);
    // (the same in every lane, which the compiler cannot see)
    const int h = __builtin_amdgcn_readfirstlane(pc.h);
    const int m0 = __builtin_amdgcn_readfirstlane(pc.rt * MT);
    const int k0 = __builtin_amdgcn_readfirstlane(pc.k0);
    const int k1 = __builtin_amdgcn_readfirstlane(pc.k1);
    tiles_piece<C>(a, ws, rq, b, h, m0, k0, k1, 2 * run.run + (k0 == 0),
                   tiles, odd_s);
    note_piece(a, ws, run, rq, pc, join);
    run.u += pc.k1 - pc.k0;
  }
  if (threadIdx.x == 0 && ws.row_tiles == 0) store_meta(ws, run.run, join);
}

}  // namespace pct
