// Gradient of the layer output with respect to the gates: one dot product of d terms per
// pick (formulas in include/lc_moe_train.h).
#include "train.h"
#include "topk.h"

namespace lcm {

template <typename Tp>
__device__ __forceinline__ float dot_chunk(const Tp* a, const Tp* b, float acc);
template <>
__device__ __forceinline__ float dot_chunk<bf16_t>(const bf16_t* a, const bf16_t* b, float acc) {
  const uint4 p = *reinterpret_cast<const uint4*>(a), q = *reinterpret_cast<const uint4*>(b);
  const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), acc);
    acc = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), acc);
  }
  return acc;
}
template <>
__device__ __forceinline__ float dot_chunk<float>(const float* a, const float* b, float acc) {
  const float4 p = *reinterpret_cast<const float4*>(a), q = *reinterpret_cast<const float4*>(b);
  acc = fmaf(p.x, q.x, acc);
  acc = fmaf(p.y, q.y, acc);
  acc = fmaf(p.z, q.z, acc);
  return fmaf(p.w, q.w, acc);
}

// One wave per pick.
template <typename Tp>
__global__ __launch_bounds__(256) void gate_backward_kernel(const Tp* __restrict__ x, const Tp* __restrict__ rows,
                                                            int num_rows, const int32_t* __restrict__ slot_row,
                                                            const Tp* __restrict__ dy, float* __restrict__ dgate,
                                                            int picks, int d, int K) {
  constexpr int V = 16 / sizeof(Tp);
  const int i = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (i >= picks) return;
  const int t = i / K, r = slot_row[i];
  float acc = 0.f;
  if (r < num_rows) {
    const Tp* a = r < 0 ? x + size_t(t) * d : rows + size_t(r) * d;
    const Tp* b = dy + size_t(t) * d;
    for (int c = lane * V; c < d; c += 64 * V) acc = dot_chunk<Tp>(a + c, b + c, acc);
  }
  acc = __ockl_wfred_add_f32(acc);
  if (lane == 0) dgate[i] = acc;
}

hipError_t launch_gate_backward(const lc_moe_shape& s, const void* x, const void* rows, int num_rows,
                                const int32_t* slot_row, const void* dy, float* dgate, hipStream_t st) {
  const int picks = s.T * s.K;
  const dim3 grid(unsigned((picks + 3) / 4));
  if (s.dtype == LC_MOE_BF16)
    hipLaunchKernelGGL(gate_backward_kernel<bf16_t>, grid, dim3(256), 0, st, static_cast<const bf16_t*>(x),
                       static_cast<const bf16_t*>(rows), num_rows, slot_row, static_cast<const bf16_t*>(dy), dgate,
                       picks, s.d, s.K);
  else
    hipLaunchKernelGGL(gate_backward_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(x),
                       static_cast<const float*>(rows), num_rows, slot_row, static_cast<const float*>(dy), dgate,
                       picks, s.d, s.K);
  return hipGetLastError();
}

}  // namespace lcm
