// C-ABI entry points of the block operators: argument checks, workspace carving and the launch
// sequence.  Every argument's meaning is documented in include/lc_moe_block.h.
#include <cfloat>
#include <cmath>

#include "block.h"
#include "checks.h"

using namespace lcm;

namespace {

lc_moe_status check_space(const void* ws, size_t bytes, size_t need) {
  if (!ws) return LC_MOE_E_NULLPTR;
  if (!aligned16(ws)) return LC_MOE_E_ALIGN;
  return bytes < need ? LC_MOE_E_WORKSPACE : LC_MOE_OK;
}

lc_moe_status check_gating(const lc_moe_shape& s, const lc_moe_gating* g) {
  if (!g) return LC_MOE_E_NULLPTR;
  const int E = s.N + s.Z;
  if (s.K > kMaxPicks || (g->score != LC_MOE_SOFTMAX && g->score != LC_MOE_SIGMOID) || !std::isfinite(g->scale))
    return LC_MOE_E_SHAPE;
  if (g->groups < 1 || g->groups > kMaxGroups || E % g->groups != 0) return LC_MOE_E_SHAPE;
  const int size = E / g->groups;
  if (g->top_groups < 1 || g->top_groups > g->groups || s.K > g->top_groups * size) return LC_MOE_E_SHAPE;
  if (g->group_rank < 1 || g->group_rank > 2 || g->group_rank > size) return LC_MOE_E_SHAPE;
  return LC_MOE_OK;
}

lc_moe_status check_norm(int T, int d, int dtype, const lc_moe_norm* n) {
  if (!n) return LC_MOE_E_NULLPTR;
  if (dtype != LC_MOE_F32 && dtype != LC_MOE_BF16) return LC_MOE_E_DTYPE;
  if (T < 0 || T >= (1 << 24) || d < 1 || d > kNormMaxD || d % (dtype == LC_MOE_BF16 ? 8 : 4) != 0)
    return LC_MOE_E_SHAPE;
  if (!(n->eps >= FLT_MIN && n->eps <= FLT_MAX) || !std::isfinite(n->residual_scale) || !std::isfinite(n->block_scale))
    return LC_MOE_E_SHAPE;
  if (n->gate_kind != LC_MOE_GATE_NONE && n->gate_kind != LC_MOE_GATE_CHANNEL && n->gate_kind != LC_MOE_GATE_TOKEN)
    return LC_MOE_E_SHAPE;
  return LC_MOE_OK;
}

constexpr int kMaxDim = 1 << 24;
bool matrix_ok(int rows, int cols) {
  if (rows < 1 || cols < 1 || rows >= kMaxDim || cols >= kMaxDim) return false;
  const size_t rp = (size_t(rows) + 255) / 256 * 256, cp = (size_t(cols) + 127) / 128 * 128;
  return rp * cp <= size_t(1) << 37;
}
// The product's operands exist, and its tiles can be counted.
bool matmul_ok(int M, int N, int K) {
  const int m = M < 1 ? 1 : M;
  return N >= 8 && N % 8 == 0 && matrix_ok(m, K) && matrix_ok(N, K) && matrix_ok(m, N);
}
lc_moe_status check_overlap(const void* a, const void* b) { return a && a == b ? LC_MOE_E_SHAPE : LC_MOE_OK; }

struct LinearPlan {
  LinearFewPlan few;
  size_t x, mm, total;  // mm 0: few
};
LinearPlan plan_linear(int T, int k, int n) {
  LinearPlan p{};
  p.x = 0;
  p.few = plan_linear_few(T, k, n);
  if (linear_few(p.few, T, k, n)) {
    p.total = p.few.total;
    return p;
  }
  p.mm = align256(plan_fp8_mat(T, k).total);
  p.total = p.mm + plan_matmul_fp8(T, n, k).total;
  return p;
}
bool linear_ok(int T, int k, int n) {
  return T >= 0 && k >= 8 && k % 8 == 0 && matmul_ok(T, n, k);
}
struct LinearBwPlan {
  LinearFewPlan few;  // total 0: not taken
  size_t dy, dyt, xt, mm, total;
};
LinearBwPlan plan_linear_backward(int T, int k, int n) {
  LinearBwPlan p{};
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  p.dy = take(plan_fp8_mat(T, n).total);
  p.dyt = take(plan_fp8_mat(n, T).total);
  p.xt = take(plan_fp8_mat(k, T).total);
  const size_t a = plan_matmul_fp8(T, k, n).total, b = plan_matmul_fp8(n, k, T).total;
  p.mm = take(a > b ? a : b);
  p.few = plan_linear_few(T, n, k);  // dx alone: the linear layer of the transpose
  if (!linear_few(p.few, T, n, k)) p.few.total = 0;
  if (p.few.total > o) o = p.few.total;
  p.total = o;
  return p;
}
bool linear_backward_ok(int T, int k, int n) {
  if (T < 0 || T >= kMaxDim || n < 8 || n % 8 != 0 || k < 8 || k % 8 != 0) return false;
  const int t = T < 1 ? 1 : T;
  return matrix_ok(t, n) && matrix_ok(n, t) && matrix_ok(k, t) && matmul_ok(t, k, n) && matmul_ok(n, k, t);
}

__global__ void zero_kernel(uint4* __restrict__ p, size_t n16) {
  for (size_t i = size_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n16; i += size_t(gridDim.x) * blockDim.x)
    p[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

extern "C" {

lc_moe_status lc_moe_select(const lc_moe_shape* shape, const lc_moe_gating* gating, const float* logits,
                            const float* bias, const uint8_t* token_mask, int32_t* topk_idx, float* topk_gate,
                            hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  LCM_CHECK(check_gating(*shape, gating));
  LCM_CHECK(check_ptr(logits));
  LCM_CHECK(check_ptr(bias, true));
  LCM_CHECK(check_ptr(token_mask, true));
  LCM_CHECK(check_ptr(topk_idx));
  LCM_CHECK(check_ptr(topk_gate));
  LCM_LAUNCH(launch_select(*shape, *gating, logits, bias, token_mask, topk_idx, topk_gate, stream));
  return LC_MOE_OK;
}

lc_moe_status lc_moe_route_select(const lc_moe_shape* shape, const lc_moe_gating* gating, const void* x,
                                  const float* w_router, const float* bias, const uint8_t* token_mask,
                                  int32_t* topk_idx, float* topk_gate, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  LCM_CHECK(check_gating(*shape, gating));
  LCM_CHECK(check_ptr(x));
  LCM_CHECK(check_ptr(w_router));
  LCM_CHECK(check_ptr(bias, true));
  LCM_CHECK(check_ptr(token_mask, true));
  LCM_CHECK(check_ptr(topk_idx));
  LCM_CHECK(check_ptr(topk_gate));
  const WsPlan p = plan_workspace(*shape);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  float* logits = at<float>(workspace, p.logits);
  LCM_LAUNCH(launch_router_logits(*shape, x, w_router, at<bf16_t>(workspace, p.wsplit), logits,
                                  at<float>(workspace, p.rpart), stream));
  LCM_LAUNCH(launch_select(*shape, *gating, logits, bias, token_mask, topk_idx, topk_gate, stream));
  return LC_MOE_OK;
}

lc_moe_status lc_moe_select_backward(const lc_moe_shape* shape, const lc_moe_gating* gating, const float* logits,
                                     const int32_t* topk_idx, const float* dgate, const float* dlogits_aux,
                                     float* dlogits, hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  if (!gating) return LC_MOE_E_NULLPTR;
  if (shape->K > kMaxPicks || (gating->score != LC_MOE_SOFTMAX && gating->score != LC_MOE_SIGMOID) ||
      !std::isfinite(gating->scale))
    return LC_MOE_E_SHAPE;
  LCM_CHECK(check_ptr(logits));
  LCM_CHECK(check_ptr(topk_idx));
  LCM_CHECK(check_ptr(dgate));
  LCM_CHECK(check_ptr(dlogits_aux, true));
  LCM_CHECK(check_ptr(dlogits));
  LCM_LAUNCH(launch_select_backward(*shape, *gating, logits, topk_idx, dgate, dlogits_aux, dlogits, stream));
  return LC_MOE_OK;
}

lc_moe_status lc_moe_block_norm(int32_t T, int32_t d, int32_t dtype, const lc_moe_norm* norm, const void* x,
                                const void* y, const float* gate, const float* w_post, const float* w_pre, void* h,
                                void* z, hipStream_t stream) {
  LCM_CHECK(check_norm(T, d, dtype, norm));
  if (T == 0) return LC_MOE_OK;
  LCM_CHECK(check_ptr(x));
  LCM_CHECK(check_ptr(y, true));
  LCM_CHECK(check_ptr(gate, norm->gate_kind == LC_MOE_GATE_NONE));
  LCM_CHECK(check_ptr(w_post, true));
  LCM_CHECK(check_ptr(w_pre, !z));
  LCM_CHECK(check_ptr(h, true));
  LCM_CHECK(check_ptr(z, true));
  if (!y && (w_post || norm->gate_kind != LC_MOE_GATE_NONE)) return LC_MOE_E_NULLPTR;
  LCM_CHECK(check_overlap(h, z));
  if (!h && !z) return LC_MOE_OK;
  LCM_LAUNCH(launch_block_norm(T, d, dtype, *norm, x, y, gate, w_post, w_pre, h, z, stream));
  return LC_MOE_OK;
}

size_t lc_moe_block_norm_backward_workspace_size(int32_t T, int32_t d, int32_t dtype) {
  const lc_moe_norm n{1.f, 1.f, 1.f, LC_MOE_GATE_NONE};
  if (check_norm(T, d, dtype, &n) != LC_MOE_OK) return 0;
  return plan_norm_backward(T, d, dtype).total;
}

lc_moe_status lc_moe_block_norm_backward(int32_t T, int32_t d, int32_t dtype, const lc_moe_norm* norm, const void* h,
                                         const void* dh, const void* dz, const void* y, const float* gate,
                                         const float* w_post, const float* w_pre, void* dx, void* dy, float* dw_pre,
                                         float* dw_post, float* dgate, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
  LCM_CHECK(check_norm(T, d, dtype, norm));
  LCM_CHECK(check_ptr(h, T == 0));
  LCM_CHECK(check_ptr(dh, true));
  LCM_CHECK(check_ptr(dz, true));
  LCM_CHECK(check_ptr(y, true));
  LCM_CHECK(check_ptr(gate, norm->gate_kind == LC_MOE_GATE_NONE || T == 0));
  LCM_CHECK(check_ptr(w_post, true));
  LCM_CHECK(check_ptr(w_pre, !dz));
  LCM_CHECK(check_ptr(dx, true));
  LCM_CHECK(check_ptr(dy, true));
  LCM_CHECK(check_ptr(dw_pre, true));
  LCM_CHECK(check_ptr(dw_post, true));
  LCM_CHECK(check_ptr(dgate, true));
  if (T > 0 && !y && (dy || dgate || dw_post || w_post || norm->gate_kind != LC_MOE_GATE_NONE)) return LC_MOE_E_NULLPTR;
  if (T > 0 && dw_post && !w_post) return LC_MOE_E_NULLPTR;
  if (dgate && norm->gate_kind == LC_MOE_GATE_NONE) return LC_MOE_E_SHAPE;
  LCM_CHECK(check_overlap(dx, dy));
  const NormBwPlan p = plan_norm_backward(T, d, dtype);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_LAUNCH(launch_block_norm_backward(T, d, dtype, *norm, p, workspace, h, dh, dz, y, gate, w_post, w_pre, dx, dy,
                                        dw_pre, dw_post, dgate, stream));
  return LC_MOE_OK;
}

size_t lc_moe_fp8_matrix_size(int32_t rows, int32_t cols) {
  return matrix_ok(rows, cols) ? plan_fp8_mat(rows, cols).total : 0;
}

lc_moe_status lc_moe_quantize_matrix(const void* x, int32_t rows, int32_t cols, int32_t block_rows, void* out,
                                     void* out_t, hipStream_t stream) {
  if (rows < 0 || cols < 8 || cols % 8 != 0 || (block_rows != 1 && block_rows != 128)) return LC_MOE_E_SHAPE;
  if (!matrix_ok(rows < 1 ? 1 : rows, cols) || (out_t && !matrix_ok(cols, rows < 1 ? 1 : rows))) return LC_MOE_E_SHAPE;
  if (rows == 0) return LC_MOE_OK;
  LCM_CHECK(check_ptr(x));
  LCM_CHECK(check_ptr(out, true));
  LCM_CHECK(check_ptr(out_t, true));
  LCM_CHECK(check_overlap(out, out_t));
  if (!out && !out_t) return LC_MOE_OK;
  LCM_LAUNCH(launch_quantize_matrix(x, rows, cols, block_rows, out, out_t, stream));
  return LC_MOE_OK;
}

size_t lc_moe_matmul_fp8_workspace_size(int32_t M, int32_t N, int32_t K) {
  return M >= 0 && matmul_ok(M, N, K) ? plan_matmul_fp8(M < 1 ? 1 : M, N, K).total : 0;
}

lc_moe_status lc_moe_matmul_fp8(int32_t M, int32_t N, int32_t K, const void* a, const void* b, const void* add,
                                void* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (M < 0 || !matmul_ok(M, N, K)) return LC_MOE_E_SHAPE;
  if (M == 0) return LC_MOE_OK;
  LCM_CHECK(check_ptr(a));
  LCM_CHECK(check_ptr(b));
  LCM_CHECK(check_ptr(add, true));
  LCM_CHECK(check_ptr(out));
  const MatmulPlan p = plan_matmul_fp8(M, N, K);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_LAUNCH(launch_matmul_fp8(M, N, K, p, workspace, a, b, add, out, stream));
  return LC_MOE_OK;
}

size_t lc_moe_linear_fp8_workspace_size(int32_t T, int32_t k, int32_t n) {
  return linear_ok(T, k, n) ? plan_linear(T < 1 ? 1 : T, k, n).total : 0;
}

lc_moe_status lc_moe_linear_fp8(int32_t T, int32_t k, int32_t n, const void* x, const void* w, const void* add,
                                void* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!linear_ok(T, k, n)) return LC_MOE_E_SHAPE;
  if (T == 0) return LC_MOE_OK;
  LCM_CHECK(check_ptr(x));
  LCM_CHECK(check_ptr(w));
  LCM_CHECK(check_ptr(add, true));
  LCM_CHECK(check_ptr(y));
  const LinearPlan p = plan_linear(T, k, n);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_CHECK(check_overlap(x, y));
  if (p.mm == 0) {
    LCM_LAUNCH(launch_linear_few(T, k, n, p.few, workspace, x, w, add, y, stream));
    return LC_MOE_OK;
  }
  void* xq = at<void>(workspace, p.x);
  LCM_LAUNCH(launch_quantize_matrix(x, T, k, 1, xq, nullptr, stream));
  LCM_LAUNCH(launch_matmul_fp8(T, n, k, plan_matmul_fp8(T, n, k), at<char>(workspace, p.mm), xq, w, add, y, stream));
  return LC_MOE_OK;
}

size_t lc_moe_linear_fp8_backward_workspace_size(int32_t T, int32_t k, int32_t n) {
  return linear_backward_ok(T, k, n) ? plan_linear_backward(T < 1 ? 1 : T, k, n).total : 0;
}

lc_moe_status lc_moe_linear_fp8_backward(int32_t T, int32_t k, int32_t n, const void* dy, const void* x,
                                         const void* w_t, const void* dx_add, void* dx, void* dw, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
  if (!linear_backward_ok(T, k, n)) return LC_MOE_E_SHAPE;
  LCM_CHECK(check_ptr(dw, true));
  if (T == 0) {
    if (!dw) return LC_MOE_OK;
    const size_t n16 = size_t(n) * k / 8;
    zero_kernel<<<dim3(unsigned(n16 / 256 + 1 < 2048 ? n16 / 256 + 1 : 2048)), dim3(256), 0, stream>>>(
        static_cast<uint4*>(dw), n16);
    return hipGetLastError() == hipSuccess ? LC_MOE_OK : LC_MOE_E_DEVICE;
  }
  LCM_CHECK(check_ptr(dy));
  LCM_CHECK(check_ptr(x, !dw));
  LCM_CHECK(check_ptr(w_t, !dx));
  LCM_CHECK(check_ptr(dx_add, true));
  LCM_CHECK(check_ptr(dx, true));
  const LinearBwPlan p = plan_linear_backward(T, k, n);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_CHECK(check_overlap(dy, dx));
  if (!dx && !dw) return LC_MOE_OK;
  void *dyq = at<void>(workspace, p.dy), *dyt = at<void>(workspace, p.dyt), *xt = at<void>(workspace, p.xt);
  char* mm = at<char>(workspace, p.mm);
  if (!dw && p.few.total) {
    LCM_LAUNCH(launch_linear_few(T, n, k, p.few, workspace, dy, w_t, dx_add, dx, stream));
    return LC_MOE_OK;
  }
  if (!dw) {
    LCM_LAUNCH(launch_quantize_matrix(dy, T, n, 1, dyq, nullptr, stream));
    LCM_LAUNCH(launch_matmul_fp8(T, k, n, plan_matmul_fp8(T, k, n), mm, dyq, w_t, dx_add, dx, stream));
    return LC_MOE_OK;
  }
  LCM_LAUNCH(launch_quantize_gradients(dy, T, n, dx ? dyq : nullptr, dyt, x, k, xt, stream));
  if (dx)
    LCM_LAUNCH(launch_matmul_gradients(T, k, n, mm, dyq, w_t, dx_add, dx, dyt, xt, dw, stream));
  else
    LCM_LAUNCH(launch_matmul_fp8(n, k, T, plan_matmul_fp8(n, k, T), mm, dyt, xt, nullptr, dw, stream));
  return LC_MOE_OK;
}

}  // extern "C"
