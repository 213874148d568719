// Gradient of the layer output with respect to the gates: one dot product of d terms per
// pick (formulas in include/lc_moe_train.h).  Bound by reading the FFN rows once.  A wave takes
// up to three picks of a token, whose rows it reads beside one another and against the same
// piece of dy, two pieces in flight: T = 16384, d = 6144, K = 12 (2.0 GB) takes 331 us, 6.1 TB/s;
// one pick a wave 361 (366 with one piece), two 337, four 333, six 333.
#include "train.h"
#include "topk.h"

namespace lcm {

// acc + the products of 16 bytes of two rows
template <typename Tp>
__device__ __forceinline__ float dot16(const uint4& p, const uint4& q, float acc) {
  const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(Tp) == 2) {
      acc = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), acc);
      acc = fmaf(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), acc);
    } else {
      acc = fmaf(__uint_as_float(u[i]), __uint_as_float(v[i]), acc);
    }
  }
  return acc;
}

// One wave per P picks of a token; U pieces of 64 x 16 bytes of every row in flight.
template <typename Tp, int P, int U>
__global__ __launch_bounds__(256) void gate_backward_kernel(const Tp* __restrict__ x, const Tp* __restrict__ rows,
                                                            int num_rows, const int32_t* __restrict__ slot_row,
                                                            const Tp* __restrict__ dy, float* __restrict__ dgate,
                                                            int waves, int d, int K, int groups) {
  constexpr int V = 16 / sizeof(Tp);
  const int w = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (w >= waves) return;
  const int t = w / groups, k0 = (w - t * groups) * P;
  const Tp* b = dy + size_t(t) * d;
  const Tp* a[P];
  float acc[P];
  bool none[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    // picks past the last repeat it; rows out of range read x and give 0
    const int k = k0 + i < K ? k0 + i : K - 1;
    const int r = __builtin_amdgcn_readfirstlane(slot_row[size_t(t) * K + k]);
    none[i] = r >= num_rows;
    a[i] = r < 0 || r >= num_rows ? x + size_t(t) * d : rows + size_t(r) * d;
    acc[i] = 0.f;
  }
  int c = lane * V;
  for (; c + (U - 1) * 64 * V < d; c += U * 64 * V) {
    uint4 q[U], p[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u] = *reinterpret_cast<const uint4*>(b + c + u * 64 * V);
#pragma unroll
      for (int i = 0; i < P; ++i) p[u][i] = *reinterpret_cast<const uint4*>(a[i] + c + u * 64 * V);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] = dot16<Tp>(p[u][i], q[u], acc[i]);
  }
  for (; c < d; c += 64 * V) {
    const uint4 q = *reinterpret_cast<const uint4*>(b + c);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = dot16<Tp>(*reinterpret_cast<const uint4*>(a[i] + c), q, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float v = __ockl_wfred_add_f32(acc[i]);
    if (lane == 0 && k0 + i < K) dgate[size_t(t) * K + k0 + i] = none[i] ? 0.f : v;
  }
}

template <typename Tp, int P>
static void launch(const lc_moe_shape& s, const void* x, const void* rows, int num_rows, const int32_t* slot_row,
                   const void* dy, float* dgate, hipStream_t st) {
  const int groups = (s.K + P - 1) / P, waves = s.T * groups;
  hipLaunchKernelGGL((gate_backward_kernel<Tp, P, 2>), dim3(unsigned((waves + 3) / 4)), dim3(256), 0, st,
                     static_cast<const Tp*>(x), static_cast<const Tp*>(rows), num_rows, slot_row,
                     static_cast<const Tp*>(dy), dgate, waves, s.d, s.K, groups);
}

hipError_t launch_gate_backward(const lc_moe_shape& s, const void* x, const void* rows, int num_rows,
                                const int32_t* slot_row, const void* dy, float* dgate, hipStream_t st) {
  const bool bf = s.dtype == LC_MOE_BF16;
#define LCM_GATE(P)                                                                            \
  bf ? launch<bf16_t, P>(s, x, rows, num_rows, slot_row, dy, dgate, st)                       \
     : launch<float, P>(s, x, rows, num_rows, slot_row, dy, dgate, st)
  if (s.K == 1) LCM_GATE(1);
  else if (s.K == 2) LCM_GATE(2);
  else LCM_GATE(3);
#undef LCM_GATE
  return hipGetLastError();
}

}  // namespace lcm
