// k_attend.hip -- tree attention: the choice of tile, the workspace and the
// join of row tiles whose keys were split over workgroups.
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

namespace {

constexpr int kCus = 256;  // compute units of an MI355X

int padded(int D) {
  return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256;
}

struct WsLayout {
  size_t o, ml, meta, total;
};

AttendPlan plan_attend(int batch, int N, int64_t cap, int Hq, int Hkv, int D) {
  AttendPlan p{};
  p.dp = padded(D);
  // the smallest row tile that holds a request's rows of one head
  const int64_t M = (int64_t)(N + 1) * (Hq / Hkv);
  p.shared = M > 32;
  p.nt = M <= 16 || (p.shared && M <= 64) ? 1 : 2;
  p.mt = 16 * p.nt * (p.shared ? 4 : 1);
  p.n_wg = kCus * (p.dp <= 128 ? 2 : 1);
  return p;
}

WsLayout layout(const AttendPlan& p) {
  WsLayout w{};
  const size_t rows = (size_t)2 * p.n_wg * p.mt;
  w.o = 0;
  w.ml = rows * p.dp * sizeof(float);
  w.meta = w.ml + rows * sizeof(float2);
  w.total = w.meta + (size_t)p.n_wg * sizeof(int4);
  return w;
}

}  // namespace

// One workgroup per (run, quarter of the row tile) adds up the sums of a row
// tile that starts in this run and ends in a later one, in order of runs
// within each of PG groups of runs and then over the groups:
//   m = max_w m_w, out = sum_w 2^(m_w - m) O_w / sum_w 2^(m_w - m) l_w.
constexpr int kJoinThreads = 1024;

template <bool BF16>
__device__ __forceinline__ uint32_t round_pair(float x, float y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {x, y};
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void attend_join_kernel(
    AttendArgs a, AttendPlan p, AttendWs ws) {
  __shared__ float4 acc_s[kJoinThreads];
  __shared__ float2 ml_s[kJoinThreads];
  const PageGeom& g = a.g;
  const int run = blockIdx.x;
  const int4 seg = ws.meta[run];
  if (seg.w < 0) return;
  const int b = seg.x, h = seg.y, rt = seg.z;
  const int runs = seg.w - run + 1;
  const int n = g.n_nodes ? clamp_nodes(g.n_nodes[b], g.N) : g.N;
  const int M = (n + 1) * a.G;
  const int tid = threadIdx.x;
  // LR threads per row (4 elements each), rows at a time, groups of runs
  const int LR = p.dp <= 64 ? 16 : p.dp <= 128 ? 32 : 64;
  const int quarter = p.mt / 4;
  const int rows = min(quarter, kJoinThreads / LR);
  const int PG = kJoinThreads / (LR * rows);
  const int c = tid % LR, r_in = tid / LR % rows, pg = tid / (LR * rows);
  const bool on = 4 * c < g.D;
  for (int r0 = 0; r0 < quarter; r0 += rows) {
    const int r = blockIdx.y * quarter + r0 + r_in;
    const int m = rt * p.mt + r;
    const bool live = m < M && on;
    float top = neg_inf(), sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      constexpr int U = 8;  // runs in flight
      for (int x0 = pg; x0 < runs; x0 += U * PG) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int x = x0 + k * PG;
          ml[k] = make_float2(neg_inf(), 0.f);
          o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x < runs) {
            const int64_t row =
                (int64_t)(2 * (run + x) + (x == 0 ? 1 : 0)) * p.mt + r;
            ml[k] = ws.ml[row];
            o[k] = reinterpret_cast<const float4*>(ws.o + row * p.dp)[c];
          }
        }
        float t2 = top;
#pragma unroll
        for (int k = 0; k < U; ++k) t2 = fmaxf(t2, ml[k].x);
        const float f0 =
            t2 == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(top - t2);
        sum *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
        top = t2;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (x0 + k * PG >= runs) continue;
          const float f =
              t2 == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml[k].x - t2);
          sum += f * ml[k].y;
          acc.x += f * o[k].x;
          acc.y += f * o[k].y;
          acc.z += f * o[k].z;
          acc.w += f * o[k].w;
        }
      }
    }
    if (PG > 1) {
      __syncthreads();
      acc_s[tid] = acc;
      ml_s[tid] = make_float2(top, sum);
      __syncthreads();
      if (pg == 0) {
        const int step = LR * rows;
        float t2 = neg_inf();
        for (int y = 0; y < PG; ++y) t2 = fmaxf(t2, ml_s[tid + y * step].x);
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y = 0; y < PG; ++y) {
          const float2 q = ml_s[tid + y * step];
          const float4 v = acc_s[tid + y * step];
          const float f =
              t2 == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(q.x - t2);
          sum += f * q.y;
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        top = t2;
      }
    }
    if (live && pg == 0) {
      const int i = m / a.G;
      const int64_t row =
          ((int64_t)b * (g.N + 1) + i) * a.Hq + h * a.G + (m - i * a.G);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * g.D)[c] =
          make_uint2(round_pair<BF16>(acc.x * inv, acc.y * inv),
                     round_pair<BF16>(acc.z * inv, acc.w * inv));
      if (a.lse && c == 0)
        a.lse[row] = sum == 0.f ? neg_inf()
                                : (top + __builtin_log2f(sum)) * (float)kLn2;
    }
  }
}

size_t tree_attention_workspace(const pct_cache_shape& sh) {
  return layout(plan_attend(sh.batch, sh.N,
                            (int64_t)sh.max_pages * sh.page_size, sh.Hq,
                            sh.Hkv, sh.D))
      .total;
}

hipError_t launch_tree_attention(const AttendArgs& a, void* workspace,
                                 hipStream_t s) {
  const PageGeom& g = a.g;
  const AttendPlan p = plan_attend(
      g.batch, g.N, (int64_t)g.max_pages << g.shift, a.Hq, g.Hkv, g.D);
  const WsLayout w = layout(p);
  char* base = static_cast<char*>(workspace);
  AttendWs ws{reinterpret_cast<float*>(base + w.o),
              reinterpret_cast<float2*>(base + w.ml),
              reinterpret_cast<int4*>(base + w.meta)};
  hipError_t e;
  {
    ProfScope ps(PROF_ATTEND, (int64_t)g.batch * (g.N + 1), s);
    switch (p.dp) {
      case 64: e = launch_attend_d64(a, p, ws, s); break;
      case 96: e = launch_attend_d96(a, p, ws, s); break;
      case 128: e = launch_attend_d128(a, p, ws, s); break;
      case 192: e = launch_attend_d192(a, p, ws, s); break;
      default: e = launch_attend_d256(a, p, ws, s); break;
    }
  }
  if (e != hipSuccess) return e;
  ProfScope ps(PROF_JOIN, (int64_t)g.batch * (g.N + 1), s);
  const dim3 grid(p.n_wg, 4);
  if (a.bf16)
    hipLaunchKernelGGL(attend_join_kernel<true>, grid, dim3(kJoinThreads), 0,
                       s, a, p, ws);
  else
    hipLaunchKernelGGL(attend_join_kernel<false>, grid, dim3(kJoinThreads), 0,
                       s, a, p, ws);
  return hipGetLastError();
}

}  // namespace pct
