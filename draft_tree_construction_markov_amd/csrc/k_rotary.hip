// k_rotary.hip -- norm and position rotation of a round's queries and keys
// on their way to the attention and into the paged cache.
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

// For a row at position p and the pair i of rotated elements (x0, x1),
//   t = p F_i mod 1 turn,  y0 = A (x0 cos t - x1 sin t),
//                          y1 = A (x1 cos t + x0 sin t),
// with F_i a fixed-point number of turns per position in units of 2^-64: the
// 64-bit product wraps at whole turns, so t is as exact at position 2^30 as
// at the first (fp32 angles are off by 2^-24 of p F_i, a whole turn at far
// positions).  Sums of squares and products are fp32; an element is rounded
// once, when it is stored.
//
// LH lanes hold a head, 4 pairs each: pairs i >= rot / 2 are the elements
// behind the rotated ones, two by two, and are not rotated.  A wave has
// 64 / LH heads at a time and goes through those of one row, the next ones on
// their way while it computes: cosines and sines are computed once per lane
// and used for all of its heads, and a pair needs no other lane.
//
// Bound by memory: 65,664 rows of 32 + 8 + 8 heads of 128, normalised and
// rotated, 1.61 GB read and written in 305 us, 5.3 TB/s (a copy of 1 GiB
// reaches 5.06).  With the partner elements read a second time and one load
// waited for at a time it was 552.  One row 3.5 us, the latency of position ->
// loads -> stores with the launch.
//
// Where a lane's pairs are: in 16 bytes (interleaved), in twice 8 (halves; rot
// a multiple of 8), or element by element (halves, other rot).
enum { kPairs = 0, kHalf = 1, kHalfOdd = 2 };

template <bool BF16>
__device__ __forceinline__ float from_bits(uint32_t b) {
  if constexpr (BF16) return __builtin_bit_cast(float, b << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

// The first and second elements of a lane's 4 pairs, from and to its 16 bytes.
template <bool BF16, int LAYOUT>
__device__ __forceinline__ void unpack_pairs(const uint4& v, float (&x)[4],
                                             float (&y)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = from_bits<BF16>(w[e] & 0xffffu);
    f[2 * e + 1] = from_bits<BF16>(w[e] >> 16);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = f[LAYOUT == kPairs ? 2 * e : e];
    y[e] = f[LAYOUT == kPairs ? 2 * e + 1 : 4 + e];
  }
}
template <bool BF16, int LAYOUT>
__device__ __forceinline__ uint4 pack_pairs(const float (&x)[4],
                                            const float (&y)[4]) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  f32x8 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[LAYOUT == kPairs ? 2 * e : e] = x[e];
    v[LAYOUT == kPairs ? 2 * e + 1 : 4 + e] = y[e];
  }
  if constexpr (BF16)
    return __builtin_bit_cast(uint4, __builtin_convertvector(v, bf16x8));
  else
    return __builtin_bit_cast(uint4, __builtin_convertvector(v, f16x8));
}

// Cosine and sine of a phase in units of 2^-64 turns, times amp.  With the
// nearest quarter turn taken off, |x| <= pi / 4 and the series to x^9 and
// x^10 end below 2^-29; what remains is the rounding of x and of the sums.
__device__ __forceinline__ void turn(uint64_t phase, float amp, float& c,
                                     float& s) {
  const uint32_t hi = (uint32_t)(phase >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(hi - (quarter << 30)) *
                  (float)(6.283185307179586 / 4294967296.0);
  const float y = x * x;
  float sn = 1.f / 362880.f;
  sn = __builtin_fmaf(sn, y, -1.f / 5040.f);
  sn = __builtin_fmaf(sn, y, 1.f / 120.f);
  sn = __builtin_fmaf(sn, y, -1.f / 6.f);
  sn = __builtin_fmaf(sn * y, x, x);
  float cs = -1.f / 3628800.f;
  cs = __builtin_fmaf(cs, y, 1.f / 40320.f);
  cs = __builtin_fmaf(cs, y, -1.f / 720.f);
  cs = __builtin_fmaf(cs, y, 1.f / 24.f);
  cs = __builtin_fmaf(cs, y, -0.5f);
  cs = __builtin_fmaf(cs, y, 1.f);
  const bool swap = quarter & 1;
  const float a = swap ? sn : cs, b = swap ? cs : sn;
  c = ((quarter + 1) & 2) ? -a * amp : a * amp;
  s = (quarter & 2) ? -b * amp : b * amp;
}

// sum over the LH lanes of a head
template <int LH>
__device__ __forceinline__ float head_sum(float x) {
  const auto plus = [](float x, int y) {
    return x + __builtin_bit_cast(float, y);
  };
  x = plus(x, dpp_i<kDppXor1>(__builtin_bit_cast(int, x)));
  if constexpr (LH >= 4)
    x = plus(x, dpp_i<kDppXor2>(__builtin_bit_cast(int, x)));
  if constexpr (LH == 8) x += __shfl_xor(x, 4, kWave);
  if constexpr (LH >= 16) {
    x = plus(x, dpp_i<kDppRor4>(__builtin_bit_cast(int, x)));
    x = plus(x, dpp_i<kDppRor8>(__builtin_bit_cast(int, x)));
  }
  if constexpr (LH == 32) x += __shfl_xor(x, 16, kWave);
  return x;
}

// Sum of the squares of a lane's elements.
__device__ __forceinline__ float squares(const float (&x)[4],
                                         const float (&y)[4]) {
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    sum = __builtin_fmaf(y[e], y[e], __builtin_fmaf(x[e], x[e], sum));
  return sum;
}
// Below kTiny a sum may have lost squares; elements times kDown have squares
// within the range if they themselves had none (2^128 2^-70 squared, times 256
// elements), and those times 1 / kDown if theirs were too small.
constexpr float kTiny = 0x1p-90f, kDown = 0x1p-70f;

// x or y, as values: a conditional expression of two variables is one of their
// addresses, which keeps both in memory.
template <typename T>
__device__ __forceinline__ T pick(bool c, T x, T y) {
  return c ? x : y;
}

constexpr int kRotaryThreads = 256;
constexpr int kAhead = 4;  // heads of a lane that are loaded together
constexpr int kResident = 5120;  // waves on the chip

template <int LH, bool BF16, int LAYOUT>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(
    RotaryArgs a, int splits, int per) {
  constexpr int HW = kWave / LH;  // heads of a wave at a time
  const int lane = threadIdx.x & 63;
  const int64_t wave =
      (int64_t)blockIdx.x * (kRotaryThreads / kWave) +
      __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = splits == 1       ? wave
                      : wave >> 31 == 0 ? (uint32_t)wave / (uint32_t)splits
                                        : wave / splits;
  if (row >= a.rows) return;
  const int l = lane % LH, sub = lane / LH;
  const int half = a.rot >> 1, Hq = a.Hq, Hkv = a.Hkv, D = a.D;
  const bool q_norm = a.qw != nullptr, k_norm = a.kw != nullptr;
  uint16_t* const out_row = static_cast<uint16_t*>(a.out) + row * a.os;
  uint16_t *const kc = static_cast<uint16_t*>(a.kc),
                 *const vc = static_cast<uint16_t*>(a.vc);
  const bool in = 8 * l < D;
  // units of this wave: HW query heads each, then keys, then values
  const int nq = a.q ? (Hq + HW - 1) / HW : 0;
  const int nk = a.k ? (Hkv + HW - 1) / HW : 0;
  const int u0 = (int)(wave - row * splits) * per;
  int u1 = min(u0 + per, nq + 2 * nk);
  if (u0 >= u1) return;

  // elements of the lane's pair e, and its two 8-byte pieces
  auto first_of = [&](int e) {
    const int i = 4 * l + e;
    return LAYOUT == kPairs || i >= half ? 2 * i : i;
  };
  auto second_of = [&](int e) {
    const int i = 4 * l + e;
    return LAYOUT == kPairs || i >= half ? 2 * i + 1 : i + half;
  };
  // (kHalf: behind the rotated elements a piece is two pairs; which of its
  // elements make a pair does not matter there)
  const bool pieces = LAYOUT == kHalf && 4 * l < half;
  const int lo = !in ? 0 : pieces ? 4 * l : 8 * l;
  const int hi = !in ? 4 : pieces ? 4 * l + half : 8 * l + 4;

  const uint16_t* q_row = static_cast<const uint16_t*>(a.q) + row * a.qs;
  const uint16_t* k_row = static_cast<const uint16_t*>(a.k) + row * a.ks;
  const uint16_t* v_row = static_cast<const uint16_t*>(a.v) + row * a.vs;
  // Loads are not conditional (the compiler would wait for each before the
  // next): what is past the row's end reads its last head, or the first
  // pairs, once more.
  auto load = [&](int u) __attribute__((always_inline)) {
    u = min(u, u1 - 1);
    const int kind = u < nq ? 0 : u < nq + nk ? 1 : 2;
    const int h = (kind == 0 ? u : u - nq - (kind == 2 ? nk : 0)) * HW + sub;
    const uint16_t* from =
        pick(kind == 0, q_row, pick(kind == 1, k_row, v_row)) +
        min(h, pick(kind == 0, Hq, Hkv) - 1) * D;
    if constexpr (LAYOUT == kPairs) {
      return *reinterpret_cast<const uint4*>(from + lo);
    } else if constexpr (LAYOUT == kHalf) {
      const uint2 y = *reinterpret_cast<const uint2*>(from + lo);
      const uint2 z = *reinterpret_cast<const uint2*>(from + hi);
      return make_uint4(y.x, y.y, z.x, z.y);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = from[in ? first_of(e) : e];
        w[4 + e] = from[in ? second_of(e) : e];
      }
      return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16,
                        w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
  };

  const int p = a.pos[row];
  const int64_t slot = a.k ? a.slot[row] : -1;
  uint4 next[kAhead];
#pragma unroll
  for (int x = 0; x < kAhead; ++x) next[x] = load(u0 + x);
  uint64_t f[4] = {0, 0, 0, 0};
  if (half > 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = a.freq[min(4 * l + e, half - 1)];
  }
  // norm weights of queries and keys
  float w[2][8];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float* from = y == 0 ? a.qw : a.kw;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[y][e] = 1.f;
    if (!from) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[y][e] = from[LAYOUT == kHalf ? lo + e : in ? first_of(e) : 0];
      w[y][4 + e] = from[LAYOUT == kHalf ? hi + e : in ? second_of(e) : 0];
    }
  }
  if (p < 0) return;
  if (slot < 0 || slot >= a.n_slots) u1 = min(u1, nq);
  const int64_t page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
  float cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (4 * l + e < half) turn((uint64_t)p * f[e], a.amp, cs[e], sn[e]);
  }

  for (int ub = u0; ub < u1; ub += kAhead) {
    uint4 mine[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) mine[x] = next[x];
    if (ub + kAhead < u1) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x) next[x] = load(ub + kAhead + x);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int u = ub + x;
      if (u >= u1) break;
      const int kind = u < nq ? 0 : u < nq + nk ? 1 : 2;
      const int h = (kind == 0 ? u : u - nq - (kind == 2 ? nk : 0)) * HW + sub;
      const bool live = in && h < pick(kind == 0, Hq, Hkv);
      uint16_t* to =
          kind == 0
              ? out_row + h * D
              : pick(kind == 1, kc, vc) +
                    (((page * Hkv + h) << a.shift) + off) * D;
      float x0[4], x1[4], y0[4], y1[4];
      uint4 y = mine[x];
      if (!in) y = make_uint4(0, 0, 0, 0);
      unpack_pairs<BF16, LAYOUT>(y, x0, x1);
      if (pick(kind == 0, q_norm, k_norm)) {
        float sum = head_sum<LH>(squares(x0, x1)), eps = a.eps;
        // squares out of fp32's range: elements and eps by powers of two
        const bool big = !(sum < pos_inf()), small = sum < kTiny && eps < kTiny;
        if (__ballot(big || small)) {
          const float f = big ? kDown : small ? 1.f / kDown : 1.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) x0[e] *= f, x1[e] *= f;
          sum = head_sum<LH>(squares(x0, x1));
          eps = eps * f * f;
        }
        const float inv = 1.f / __builtin_sqrtf(sum / (float)D + eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x0[e] *= inv * pick(kind == 0, w[0][e], w[1][e]);
          x1[e] *= inv * pick(kind == 0, w[0][4 + e], w[1][4 + e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool turns = 4 * l + e < half;
        const float s1 = x1[e] * sn[e], s0 = x0[e] * sn[e];
        y0[e] = turns ? __builtin_fmaf(x0[e], cs[e], -s1) : x0[e];
        y1[e] = turns ? __builtin_fmaf(x1[e], cs[e], s0) : x1[e];
      }
      if (kind != 2) y = pack_pairs<BF16, LAYOUT>(y0, y1);
      if (!live) continue;
      if constexpr (LAYOUT == kPairs) {
        reinterpret_cast<uint4*>(to)[l] = y;
      } else if constexpr (LAYOUT == kHalf) {
        *reinterpret_cast<uint2*>(to + lo) = make_uint2(y.x, y.y);
        *reinterpret_cast<uint2*>(to + hi) = make_uint2(y.z, y.w);
      } else {
        const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          to[first_of(e)] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
          to[second_of(e)] = (uint16_t)(v[2 + (e >> 1)] >> (16 * (e & 1)));
        }
      }
    }
  }
}

// Rows of a launch at most: a grid has fewer than 2^32 threads, and a row here
// 64 of them.
constexpr int64_t kLaunchRows = 1 << 25;

template <int LH, bool BF16>
hipError_t launch_rotary_lh(const RotaryArgs& a, hipStream_t s) {
  constexpr int HW = kWave / LH;
  const int units = (a.q ? (a.Hq + HW - 1) / HW : 0) +
                    (a.k ? 2 * ((a.Hkv + HW - 1) / HW) : 0);
  // a wave per row, or several while these are few
  int64_t splits = kResident / a.rows;
  splits = splits < 1 ? 1 : splits > units ? units : splits;
  const int per = (int)((units + splits - 1) / splits);
  splits = (units + per - 1) / per;
  const int64_t waves = a.rows * splits;
  const dim3 grid((unsigned)((waves + 3) / 4)), block(kRotaryThreads);
  if (a.pairs)
    hipLaunchKernelGGL((rotary_kernel<LH, BF16, kPairs>), grid, block, 0, s, a,
                       (int)splits, per);
  else if (a.rot % 8 == 0)
    hipLaunchKernelGGL((rotary_kernel<LH, BF16, kHalf>), grid, block, 0, s, a,
                       (int)splits, per);
  else
    hipLaunchKernelGGL((rotary_kernel<LH, BF16, kHalfOdd>), grid, block, 0, s,
                       a, (int)splits, per);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_rotary_type(const RotaryArgs& a, hipStream_t s) {
  if (a.D <= 16) return launch_rotary_lh<2, BF16>(a, s);
  if (a.D <= 32) return launch_rotary_lh<4, BF16>(a, s);
  if (a.D <= 64) return launch_rotary_lh<8, BF16>(a, s);
  if (a.D <= 128) return launch_rotary_lh<16, BF16>(a, s);
  return launch_rotary_lh<32, BF16>(a, s);
}

hipError_t launch_cache_rotary(const RotaryArgs& all, hipStream_t s) {
  for (int64_t row = 0; row < all.rows; row += kLaunchRows) {
    RotaryArgs a = all;
    a.rows = all.rows - row < kLaunchRows ? all.rows - row : kLaunchRows;
    const auto from = [&](const void* x, int64_t stride) {
      return x ? static_cast<const uint16_t*>(x) + row * stride : nullptr;
    };
    a.q = from(all.q, all.qs);
    a.k = from(all.k, all.ks);
    a.v = from(all.v, all.vs);
    if (all.out) a.out = static_cast<uint16_t*>(all.out) + row * all.os;
    a.pos = all.pos + row;
    if (all.slot) a.slot = all.slot + row;
    const hipError_t e = a.bf16 ? launch_rotary_type<true>(a, s)
                                : launch_rotary_type<false>(a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace pct
