// Internal definitions of the block operators (include/lc_moe_block.h).
#pragma once

#include <type_traits>

#include "common.h"
#include "lc_moe_block.h"

namespace lcm {

// ---- choice of experts -----------------------------------------------------------------
constexpr int kMaxPicks = 64;   // one lane of a wavefront for each pick
constexpr int kMaxGroups = 64;  // and for each group
hipError_t launch_select(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits, const float* bias,
                         const uint8_t* mask, int32_t* idx, float* gate, hipStream_t st);
hipError_t launch_select_backward(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits,
                                  const int32_t* idx, const float* dgate, const float* aux, float* dlogits,
                                  hipStream_t st);

// ---- norms around a block ----------------------------------------------------------------
constexpr int kNormMaxD = 16384;
hipError_t launch_block_norm(int T, int d, int dtype, const lc_moe_norm& n, const void* x, const void* y,
                             const float* gate, const float* w_post, const float* w_pre, void* h, void* z,
                             hipStream_t st);
// Backward: `wgs` workgroups take the rows in turn and leave a row of partial sums each
// (part [wgs][3][d]: dw_pre, dw_post, dgate), added in order by a second kernel.
struct NormBwPlan {
  size_t part, total;
  int wgs;
};
NormBwPlan plan_norm_backward(int T, int d, int dtype);
hipError_t launch_block_norm_backward(int T, int d, int dtype, const lc_moe_norm& n, const NormBwPlan& p, void* ws,
                                      const void* h, const void* dh, const void* dz, const void* y,
                                      const float* gate, const float* w_post, const float* w_pre, void* dx, void* dy,
                                      float* dw_pre, float* dw_post, float* dgate, hipStream_t st);

// ---- block FP8 ---------------------------------------------------------------------------
struct Fp8Mat {
  size_t scales, total;  // byte offsets: codes at 0
  size_t ldc, lds;       // bytes from one row of codes, one run of scales, to the next
  int nkb;               // runs of 128 columns
};
inline Fp8Mat plan_fp8_mat(int rows, int cols) {
  Fp8Mat m{};
  m.nkb = (cols + 127) / 128;
  m.ldc = size_t(m.nkb) * 128;
  m.lds = (size_t(rows) + 255) / 256 * 256;
  m.scales = align256(size_t(rows) * m.ldc);
  m.total = m.scales + m.nkb * m.lds + 256;
  return m;
}
// Place of row r's exponent byte in its run.
__host__ __device__ __forceinline__ size_t fp8_scale_at(size_t r) {
  return (r & ~size_t(127)) + 4 * (r & 31) + (r >> 5 & 3);
}
hipError_t launch_quantize_matrix(const void* x, int rows, int cols, int block_rows, void* out, void* out_t,
                                  hipStream_t st);

// dy [T][n] by its rows (dyq, may be null) and columns (dyt), x [T][k] by its columns (xt), in blocks of
// 128 x 1.
hipError_t launch_quantize_gradients(const void* dy, int T, int n, void* dyq, void* dyt, const void* x, int k, void* xt,
                                     hipStream_t st);

struct MatmulPlan {
  size_t part, total;
  int splits, chunk;  // pieces of the reduction, runs of 128 of each
  int form;           // tile (fp8_matmul.hip)
  float us;           // what it takes, by the model
};
MatmulPlan plan_matmul_fp8(int M, int N, int K);
hipError_t launch_matmul_fp8(int M, int N, int K, const MatmulPlan& p, void* ws, const void* a, const void* b,
                             const void* add, void* out, hipStream_t st);
// out [n] = sum of `splits` pieces of n fp32 sums in order (+ add).
hipError_t launch_matmul_join(const float* part, int splits, size_t n, const bf16_t* add, bf16_t* out, hipStream_t st);
// y [T][n] = Q(x) w^T (+ add) for few tokens or small matrices, x quantised on the way, where linear_few says so.
struct LinearFewPlan {
  size_t total;
  int form, splits, chunk;  // blocks of tokens; pieces of the reduction, runs of 128 of each
  float us;                 // what it takes, by the model
};
LinearFewPlan plan_linear_few(int T, int k, int n);
bool linear_few(const LinearFewPlan& p, int T, int k, int n);
hipError_t launch_linear_few(int T, int k, int n, const LinearFewPlan& p, void* ws, const void* x, const void* w,
                             const void* add, void* y, hipStream_t st);
// A linear layer's gradients: dx [T][k] = dyq w_t^T (+ add) and dw [n][k] = dyt xt^T, in one launch where both
// take the same small tiles.  ws: room for either's plan.
hipError_t launch_matmul_gradients(int T, int k, int n, void* ws, const void* dyq, const void* w_t, const void* add,
                                   void* dx, const void* dyt, const void* xt, void* dw, hipStream_t st);

// Largest over the 16 lanes of a row, and over the four rows of a wavefront (lanes l, l + 16, ...), in every
// lane, without LDS.
__device__ __forceinline__ float max_of_row(float v) {
  const auto turned = [](float v, auto by) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), 0x120 + decltype(by)::value, 0xF, 0xF, true));
  };
  v = fmaxf(v, turned(v, std::integral_constant<int, 8>()));
  v = fmaxf(v, turned(v, std::integral_constant<int, 4>()));
  v = fmaxf(v, turned(v, std::integral_constant<int, 2>()));
  return fmaxf(v, turned(v, std::integral_constant<int, 1>()));
}
__device__ __forceinline__ uint32_t max_of_rows(uint32_t v) {
  const auto near = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // rows 0 0 2 2 and 1 1 3 3
  v = near[0] > near[1] ? near[0] : near[1];
  const auto far = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // the lower half twice, and the upper
  return far[0] > far[1] ? far[0] : far[1];
}

}  // namespace lcm
