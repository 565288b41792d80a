// k_attend_join.h -- sums of an attention row that several workgroups left,
// added up.
#pragma once
#include "pct_cache.h"
#include "pct_device.h"

namespace pct {

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

struct JoinSum {
  float m, l;
  float4 o;
  __device__ __forceinline__ void scale(float m2) {
    const float f = m2 == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(m - m2);
    m = m2;
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
  }
  __device__ __forceinline__ void add(float2 ml, const float4& v) {
    const float f = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
    l += f * ml.y;
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  }
};

}  // namespace pct
