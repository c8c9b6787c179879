// Vectors of VEC storage elements as packed fp32 pairs (fp32x2 arithmetic: two
// elements per instruction), VEC = 1 padded with 0.
#pragma once

#include "gbn_common.cuh"

namespace gbn {

template <int VEC> constexpr int kPairs = (VEC + 1) / 2;

template <typename T, int VEC>
__device__ __forceinline__ void to_pairs(typename Vec<T, VEC>::raw r, f2 (&p)[kPairs<VEC>]) {
  float v[VEC];
  Vec<T, VEC>::cvt(r, v);
#pragma unroll
  for (int k = 0; k < kPairs<VEC>; ++k)
    p[k] = f2_pack(v[2 * k], 2 * k + 1 < VEC ? v[2 * k + 1] : 0.f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pairs(T* p, const f2 (&o)[kPairs<VEC>]) {
  float v[VEC];
#pragma unroll
  for (int k = 0; k < kPairs<VEC>; ++k) {
    const float2 t = f2_unpack(o[k]);
    v[2 * k] = t.x;
    if (2 * k + 1 < VEC) v[2 * k + 1] = t.y;
  }
  Vec<T, VEC>::store(p, v);
}
// Pair k of VEC floats.
template <int VEC>
__device__ __forceinline__ f2 pair_at(const float (&v)[VEC], int k) {
  return f2_pack(v[2 * k], 2 * k + 1 < VEC ? v[2 * k + 1] : 0.f);
}
__device__ __forceinline__ f2 f2_neg(f2 a) { return a ^ 0x8000000080000000ull; }

}  // namespace gbn
