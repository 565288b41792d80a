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
// LH lanes hold a head, 8 elements (16 bytes) each, so a wave has 64 / LH
// heads at a time and goes through those of one row: cosines and sines are
// computed once per lane and used for all of its heads.  The other element of
// a pair is in another lane's piece, which is loaded a second time (from the
// L1; both are whole pieces if rot / 2 is a multiple of 8).
enum { kHalf = 0, kPairs = 1, kHalfOdd = 2 };

template <bool BF16>
__device__ __forceinline__ float from_bits(uint32_t b) {
  if constexpr (BF16) return __builtin_bit_cast(float, b << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = from_bits<BF16>(w[e] & 0xffffu);
    x[2 * e + 1] = from_bits<BF16>(w[e] >> 16);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const f32x8 v = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
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
#pragma unroll
  for (int d = 1; d < LH; d <<= 1) x += __shfl_xor(x, d, kWave);
  return x;
}

constexpr int kRotaryThreads = 256;
constexpr int kAhead = 4;  // heads of a lane loaded before the first is used

template <int LH, bool BF16, int LAYOUT>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(
    RotaryArgs a, int splits, int per) {
  constexpr int HW = kWave / LH;  // heads of a wave at a time
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (kRotaryThreads / kWave) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = wave / splits;
  if (row >= a.rows) return;
  const int p = a.pos[row];
  if (p < 0) return;
  // units of this wave: the query heads in groups of HW, then keys and values
  const int nq = a.q ? (a.Hq + HW - 1) / HW : 0;
  const int nkv = a.k ? (2 * a.Hkv + HW - 1) / HW : 0;
  const int u0 = (int)(wave - row * splits) * per;
  const int u1 = min(u0 + per, nq + nkv);
  const int c = lane % LH, sub = lane / LH;
  const int chd = a.D >> 3, half = a.rot >> 1;
  const bool in = c < chd;
  // the piece with the other elements of this lane's pairs
  const int other = LAYOUT == kPairs ? c
                    : c * 8 < half   ? c + half / 8
                    : c * 8 < a.rot  ? c - half / 8
                                     : c;

  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = 8 * c + e;
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (at < a.rot) {
      if constexpr (LAYOUT == kPairs) {
        if (e % 2 == 0)
          turn((uint64_t)p * a.freq[at >> 1], a.amp, cs[e], sn[e]);
        else
          cs[e] = cs[e - 1], sn[e] = sn[e - 1];
      } else {
        turn((uint64_t)p * a.freq[at < half ? at : at - half], a.amp, cs[e],
             sn[e]);
      }
    }
  }
  // the sign of the other element's product
  if constexpr (LAYOUT == kPairs) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) sn[e] = -sn[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * c + e < half) sn[e] = -sn[e];
  }

  // the eight elements of the pairs' other halves, where these are not one
  // piece
  auto gather = [&](const uint16_t* head) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = 8 * c + e;
      const int o = at < half ? at + half : at < a.rot ? at - half : at;
      w[e] = head[o];
    }
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16,
                      w[6] | w[7] << 16);
  };
  auto weights = [&](const float* w, float (&own)[8], float (&oth)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = 8 * c + e;
      own[e] = oth[e] = 1.f;
      if (w && in) {
        own[e] = w[at];
        int o = at;
        if (LAYOUT == kPairs)
          o = at < a.rot ? at ^ 1 : at;
        else
          o = at < half ? at + half : at < a.rot ? at - half : at;
        oth[e] = w[o];
      }
    }
  };
  auto rotated = [&](const uint4& mine, const uint4& theirs, bool norm,
                     const float (&wo)[8], const float (&wt)[8]) {
    float x[8], z[8], y[8];
    unpack8<BF16>(mine, x);
    if constexpr (LAYOUT == kPairs) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = x[e ^ 1];
    } else {
      unpack8<BF16>(theirs, z);
    }
    float inv = 1.f;
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
      sum = head_sum<LH>(in ? sum : 0.f);
      inv = 1.f / __builtin_sqrtf(sum / (float)a.D + a.eps);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xo = norm ? x[e] * inv * wo[e] : x[e];
      const float xt = norm ? z[e] * inv * wt[e] : z[e];
      y[e] = 8 * c + e < a.rot ? __builtin_fmaf(xo, cs[e], xt * sn[e]) : xo;
    }
    return pack8<BF16>(y);
  };

  float wo[8], wt[8];
  if (u0 < nq) {
    weights(a.qw, wo, wt);
    const uint16_t* src = static_cast<const uint16_t*>(a.q) + row * a.qs;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.os;
    const int end = min(u1, nq);
    for (int u = u0; u < end; u += kAhead) {
      uint4 mine[kAhead], theirs[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int h = (u + x) * HW + sub;
        mine[x] = theirs[x] = make_uint4(0, 0, 0, 0);
        if (u + x < end && h < a.Hq && in) {
          const uint16_t* head = src + h * a.D;
          mine[x] = reinterpret_cast<const uint4*>(head)[c];
          if constexpr (LAYOUT == kHalf)
            theirs[x] = reinterpret_cast<const uint4*>(head)[other];
          else if constexpr (LAYOUT == kHalfOdd)
            theirs[x] = gather(head);
        }
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int h = (u + x) * HW + sub;
        if (u + x >= end) break;
        const uint4 y = rotated(mine[x], theirs[x], a.qw != nullptr, wo, wt);
        if (h < a.Hq && in) reinterpret_cast<uint4*>(dst + h * a.D)[c] = y;
      }
    }
  }
  if (u1 <= nq) return;
  const int64_t slot = a.slot[row];
  if (slot < 0 || slot >= a.n_slots) return;
  const int64_t page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
  weights(a.kw, wo, wt);
  for (int u = max(u0, nq); u < u1; u += kAhead) {
    uint4 mine[kAhead], theirs[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int j = (u + x - nq) * HW + sub;  // key heads, then value heads
      mine[x] = theirs[x] = make_uint4(0, 0, 0, 0);
      if (u + x < u1 && j < 2 * a.Hkv && in) {
        const uint16_t* head =
            j < a.Hkv
                ? static_cast<const uint16_t*>(a.k) + row * a.ks + j * a.D
                : static_cast<const uint16_t*>(a.v) + row * a.vs +
                      (j - a.Hkv) * a.D;
        mine[x] = reinterpret_cast<const uint4*>(head)[c];
        if constexpr (LAYOUT == kHalf)
          theirs[x] = reinterpret_cast<const uint4*>(head)[other];
        else if constexpr (LAYOUT == kHalfOdd)
          theirs[x] = gather(head);
      }
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int j = (u + x - nq) * HW + sub;
      if (u + x >= u1) break;
      const uint4 y = rotated(mine[x], theirs[x], a.kw != nullptr, wo, wt);
      if (j < 2 * a.Hkv && in) {
        const bool key = j < a.Hkv;
        const int h = key ? j : j - a.Hkv;
        uint4* to = reinterpret_cast<uint4*>(key ? a.kc : a.vc) +
                    (((page * a.Hkv + h) << a.shift) + off) * chd + c;
        *to = key ? y : mine[x];
      }
    }
  }
}

template <int LH, bool BF16>
hipError_t launch_rotary_lh(const RotaryArgs& a, hipStream_t s) {
  constexpr int HW = kWave / LH;
  const int units = (a.q ? (a.Hq + HW - 1) / HW : 0) +
                    (a.k ? (2 * a.Hkv + HW - 1) / HW : 0);
  // a wave per row, or several while these are few
  int64_t splits = 16384 / a.rows;
  splits = splits < 1 ? 1 : splits > units ? units : splits;
  const int per = (int)((units + splits - 1) / splits);
  splits = (units + per - 1) / per;
  const int64_t waves = a.rows * splits;
  const dim3 grid((unsigned)((waves + 3) / 4)), block(kRotaryThreads);
  if (a.pairs)
    hipLaunchKernelGGL((rotary_kernel<LH, BF16, kPairs>), grid, block, 0, s, a,
                       (int)splits, per);
  else if (a.rot % 16 == 0)
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

hipError_t launch_cache_rotary(const RotaryArgs& a, hipStream_t s) {
  return a.bf16 ? launch_rotary_type<true>(a, s)
                : launch_rotary_type<false>(a, s);
}

}  // namespace pct
