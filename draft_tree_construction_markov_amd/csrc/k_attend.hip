// k_attend.hip -- softmax attention of a round's rows over a paged
// key-value cache.  For a row with the seen positions S,
//   out = sum_{t in S} p_t v_t / sum_{t in S} p_t,  p_t = 2^(c (s_t) - m),
//   c s_t = scale * log2(e) * (q . k_t),  m = max_{t in S} c s_t,
// in one pass over the positions: m and the two sums so far are rescaled by
// 2^(m_old - m_new) when a larger score comes.
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

template <bool BF16>
__device__ __forceinline__ float elem(uint16_t b) {
  if (BF16) return bf16_bits_to_float(b);
  return (float)__builtin_bit_cast(_Float16, b);
}
template <bool BF16>
__device__ __forceinline__ uint16_t round_to(float x) {
  if (BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// One workgroup per (query head, row, request), 256 positions at a time:
// each thread scores one position, then each thread sums one element of the
// head over them.
template <bool BF16>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
  __shared__ float qv[256], pr[256], red[4];
  __shared__ int64_t vo[256];
  const PageGeom& g = a.g;
  const int hq = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  if (i > n) return;
  const int ctx = clamp_ctx(g.ctx_len[b]);
  const int cap = g.max_pages << g.shift;
  const int L = min(ctx + n + 1, cap);
  const int h = hq / a.G, D = g.D;
  const int64_t row = (int64_t)b * (g.N + 1) + i;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.qs + hq * D;
  const uint16_t* kc = static_cast<const uint16_t*>(a.kc);
  const uint16_t* vc = static_cast<const uint16_t*>(a.vc);
  const int32_t* table = g.table + (int64_t)b * g.max_pages;
  const uint64_t* mrow =
      a.mask && i > 0 ? a.mask + ((int64_t)b * g.N + i - 1) * a.words
                      : nullptr;
  if (tid < D) qv[tid] = elem<BF16>(q[tid]) * (a.scale * kLog2e);
  float m = neg_inf(), l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < L; t0 += 256) {
    __syncthreads();
    const int t = t0 + tid;
    bool see = t < L;
    if (see && t > ctx) {  // node t - ctx - 1
      const int j = t - ctx - 1;
      see = i > 0 && (mrow ? (mrow[j >> 6] >> (j & 63)) & 1 : j < i);
    }
    int64_t off = -1;
    if (see) {
      const int page = table[t >> g.shift];
      see = page >= 0 && page < g.n_pages;
      off = ((((int64_t)page * g.Hkv + h) << g.shift) +
             (t & ((1 << g.shift) - 1))) * D;
    }
    float s = neg_inf();
    if (see) {
      s = 0.f;
      const uint4* k4 = reinterpret_cast<const uint4*>(kc + off);
      for (int d = 0; d < D / 8; ++d) {
        const uint4 x = k4[d];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s += qv[8 * d + 2 * e] * elem<BF16>((uint16_t)(w[e] & 0xffff));
          s += qv[8 * d + 2 * e + 1] * elem<BF16>((uint16_t)(w[e] >> 16));
        }
      }
    }
    vo[tid] = see ? off : -1;
    float mt = wave_max(s);
    if (lane == 0) red[wave] = mt;
    __syncthreads();
    mt = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mt);
    // a tile of which nothing is seen changes nothing
    const float f = mn == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(m - mn);
    const float p = s != neg_inf() ? __builtin_amdgcn_exp2f(s - mn) : 0.f;
    m = mn;
    pr[tid] = p;
    __syncthreads();
    float ps = wave_sum(p);
    if (lane == 0) red[wave] = ps;
    l *= f;
    acc *= f;
    if (tid < D) {
      const int end = min(256, L - t0);
      for (int j = 0; j < end; ++j)
        if (vo[j] >= 0) acc += pr[j] * elem<BF16>(vc[vo[j] + tid]);
    }
    __syncthreads();
    l += red[0] + red[1] + red[2] + red[3];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN stays one)
  if (tid < D)
    static_cast<uint16_t*>(a.out)[(row * a.Hq + hq) * D + tid] =
        round_to<BF16>(acc * inv);
  if (a.lse && tid == 0)
    a.lse[row * a.Hq + hq] =
        l == 0.f ? neg_inf() : (m + log2f(l)) * (float)kLn2;
}

size_t tree_attention_workspace(const pct_cache_shape& sh) { return 16; }

hipError_t launch_tree_attention(const AttendArgs& a, void* ws,
                                 hipStream_t s) {
  ProfScope ps(PROF_ATTEND, (int64_t)a.g.batch * (a.g.N + 1), s);
  const dim3 grid(a.Hq, a.g.N + 1, a.g.batch);
  if (a.bf16)
    hipLaunchKernelGGL(attend_kernel<true>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(attend_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace pct
