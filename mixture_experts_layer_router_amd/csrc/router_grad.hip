// Backward of the router: the softmax's gradient from the gates' gradients, then the two
// products with the router weight and with the tokens (formulas in
// include/lc_moe_train.h).
#include "train.h"
#include "topk.h"

namespace lcm {

// dlogits of one token per wave; expert e in lane e % 64.  The picks' gradients are added in
// pick order: pick k is read by every lane, and the lane that holds its expert adds it.
template <int EPL>
__global__ __launch_bounds__(256) void dlogits_kernel(const float* __restrict__ logits,
                                                      const int32_t* __restrict__ idx,
                                                      const float* __restrict__ dgate, const float* aux, int T, int E,
                                                      int K, float* out) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  float v[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) v[j] = 0.f;
  if (dgate) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 64 * j;
      v[j] = e < E ? logits[size_t(t) * E + e] : -INFINITY;
      m = fmaxf(m, v[j]);
    }
    m = __ockl_wfred_max_f32(m);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      v[j] = m > -INFINITY ? expf(v[j] - m) : 0.f;
      sum += v[j];
    }
    sum = __ockl_wfred_add_f32(sum);
    const float rs = m > -INFINITY ? 1.f / sum : 0.f;
    float dp[EPL], dot = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) dp[j] = 0.f;
    for (int k = 0; k < K; ++k) {
      const int e = idx[size_t(t) * K + k];
      const float g = dgate[size_t(t) * K + k];
#pragma unroll
      for (int j = 0; j < EPL; ++j) dp[j] += e == lane + 64 * j && e < E ? g : 0.f;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      v[j] *= rs;
      dot += v[j] * dp[j];
    }
    dot = __ockl_wfred_add_f32(dot);
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] *= dp[j] - dot;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    if (e < E) out[size_t(t) * E + e] = aux ? v[j] + aux[size_t(t) * E + e] : v[j];
  }
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(bf16_t v) { return bf2f(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = f2bf(v); }

// C[M][N] = A B (+ add): A(m, k) = a[m sam + k sak], B(k, n) = b[k N + n]; 64 x 64 outputs per
// workgroup, 4 x 4 per thread, 16 reduction steps staged in LDS.
template <typename Tb, typename Tc>
__global__ __launch_bounds__(256) void router_grad_f32_kernel(const float* __restrict__ a, size_t sam, size_t sak,
                                                              const Tb* __restrict__ b, const Tc* add, Tc* c, int M,
                                                              int N, int K) {
  __shared__ float As[16][65], Bs[16][65];
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = tid; i < 64 * 16; i += 256) {
      const int k = i >> 6, r = i & 63;
      As[k][r] = m0 + r < M && k0 + k < K ? a[(m0 + r) * sam + (k0 + k) * sak] : 0.f;
      Bs[k][r] = n0 + r < N && k0 + k < K ? as_float(b[size_t(k0 + k) * N + n0 + r]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) {
        const size_t o = size_t(m) * N + n;
        put(c + o, add ? acc[i][j] + as_float(add[o]) : acc[i][j]);
      }
    }
}

template <typename Tx>
static void products(const lc_moe_shape& s, const float* dl, const void* x, const float* w, const void* add, void* dx,
                     float* dw, hipStream_t st) {
  const int E = s.N + s.Z;
  if (dx)
    hipLaunchKernelGGL((router_grad_f32_kernel<float, Tx>), dim3((s.d + 63) / 64, (s.T + 63) / 64), dim3(256), 0, st,
                       dl, size_t(E), size_t(1), w, static_cast<const Tx*>(add), static_cast<Tx*>(dx), s.T, s.d, E);
  if (dw)
    hipLaunchKernelGGL((router_grad_f32_kernel<Tx, float>), dim3((s.d + 63) / 64, (E + 63) / 64), dim3(256), 0, st,
                       dl, size_t(1), size_t(E), static_cast<const Tx*>(x), static_cast<const float*>(nullptr), dw, E,
                       s.d, s.T);
}

hipError_t launch_router_backward(const lc_moe_shape& s, const RouterBwPlan& p, void* ws, const void* x,
                                  const float* w_router, const float* logits, const int32_t* idx,
                                  const float* dgate, const float* aux, const void* dx_add, void* dx, float* dw,
                                  float* dlogits, hipStream_t st) {
  const int E = s.N + s.Z, epl = (E + 63) / 64;
  float* dl = dlogits ? dlogits : reinterpret_cast<float*>(static_cast<char*>(ws) + p.dl);
#define LCM_DL(n)                                                                                                \
  hipLaunchKernelGGL(dlogits_kernel<n>, dim3((s.T + 3) / 4), dim3(256), 0, st, logits, idx, dgate, aux, s.T, E, \
                     s.K, dl)
  if (epl <= 2) LCM_DL(2);
  else if (epl <= 4) LCM_DL(4);
  else if (epl <= 8) LCM_DL(8);
  else if (epl <= 16) LCM_DL(16);
  else if (epl <= 32) LCM_DL(32);
  else LCM_DL(64);
#undef LCM_DL
  if (s.dtype == LC_MOE_BF16) products<bf16_t>(s, dl, x, w_router, dx_add, dx, dw, st);
  else products<float>(s, dl, x, w_router, dx_add, dx, dw, st);
  return hipGetLastError();
}

}  // namespace lcm
