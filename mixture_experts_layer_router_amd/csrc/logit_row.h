// A token's row of E fp32 logits in the registers of one wavefront, shared by the balance
// loss and the router's backward.  A lane holds EPL experts: V consecutive ones (V = 4 where
// E is a multiple of 4, so that a row is read and written 16 bytes a lane; else 1) of every
// run of 64 V; element i of a lane is expert ((i / V) 64 + lane) V + i % V.
#pragma once

#include "common.h"
#include "topk.h"

namespace lcm {

template <int EPL, int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float other,
                                         float (&v)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL / V; ++j) {
    const int e = (j * 64 + lane) * V;
    if constexpr (V == 4) {
      const float4 q = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(other, other, other, other);
      v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
    } else {
      v[j] = e < E ? row[e] : other;
    }
  }
}
template <int EPL, int V>
__device__ __forceinline__ void store_row(float* row, int E, int lane, const float (&v)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL / V; ++j) {
    const int e = (j * 64 + lane) * V;
    if (e >= E) continue;
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    else
      row[e] = v[j];
  }
}

// e^x for x <= 0 within 2 ulps: x log2(e) in two floats, the hardware's base-2 exponential
// (1 ulp) of the first, and the second to first order.  Below 2^-126, and of -infinity, it is 0.
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -150.f);
  const float t = x * 1.44269502f;
  const float lo = fmaf(x, 1.44269502f, -t) + x * 1.92596299e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, lo * 0.693147182f, e);
}

// Softmax of a row held as above: v becomes e^(v - m), not yet divided; returns the largest
// logit and the sum.  m = -infinity: the row has no finite logit (v is then 0).
struct RowSum {
  float m, sum;
};
template <int EPL>
__device__ __forceinline__ RowSum softmax_row(float (&v)[EPL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = fmaxf(m, v[i]);
  m = __ockl_wfred_max_f32(m);
  float sum = 0.f;
  const float top = m > -INFINITY ? m : 0.f;  // every v is -infinity else: e^v = 0
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    v[i] = exp_neg(v[i] - top);
    sum += v[i];
  }
  return RowSum{m, __ockl_wfred_add_f32(sum)};
}

}  // namespace lcm
