// C-ABI entry points of the training operators: argument checks, workspace carving and the
// launch sequence.  Every argument's meaning is documented in include/lc_moe_train.h.
#include <cfloat>

#include "checks.h"
#include "train.h"

using namespace lcm;

namespace {

lc_moe_status check_space(const void* ws, size_t bytes, size_t need) {
  if (!ws) return LC_MOE_E_NULLPTR;
  if (!aligned16(ws)) return LC_MOE_E_ALIGN;
  return bytes < need ? LC_MOE_E_WORKSPACE : LC_MOE_OK;
}

constexpr int kMaxSeqs = 65535;

}  // namespace

extern "C" {

lc_moe_status lc_moe_forward_saved(const lc_moe_shape* shape, const void* workspace, size_t workspace_bytes,
                                   lc_moe_saved* saved) {
  LCM_CHECK(check_shape(shape));
  if (!saved) return LC_MOE_E_NULLPTR;
  const WsPlan p = plan_workspace(*shape);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  void* ws = const_cast<void*>(workspace);
  saved->logits = at<const float>(ws, p.logits);
  saved->ffn_rows = at<const char>(ws, p.ybuf);
  saved->slot_row = at<const int32_t>(ws, p.slot_row);
  saved->ffn_offsets = at<const int32_t>(ws, p.offsets);
  saved->perm_token = at<const int32_t>(ws, p.perm_token);
  return LC_MOE_OK;
}

size_t lc_moe_balance_workspace_size(const lc_moe_shape* shape, int32_t num_seqs) {
  if (check_shape(shape) != LC_MOE_OK || num_seqs < 1 || num_seqs > kMaxSeqs) return 0;
  return plan_balance(*shape, num_seqs).total;
}

lc_moe_status lc_moe_balance_loss(const lc_moe_shape* shape, const lc_moe_balance_coef* coef, const float* logits,
                                  const int32_t* topk_idx, const int32_t* seq_offsets, int32_t num_seqs,
                                  const uint8_t* token_mask, float* loss, int32_t* load, float* prob,
                                  float* dlogits, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  if (num_seqs < 1 || num_seqs > kMaxSeqs) return LC_MOE_E_SHAPE;
  if (!coef) return LC_MOE_E_NULLPTR;
  LCM_CHECK(check_ptr(logits));
  LCM_CHECK(check_ptr(topk_idx));
  LCM_CHECK(check_ptr(seq_offsets, num_seqs == 1));
  LCM_CHECK(check_ptr(token_mask, true));
  LCM_CHECK(check_ptr(loss));
  LCM_CHECK(check_ptr(load));
  LCM_CHECK(check_ptr(prob));
  LCM_CHECK(check_ptr(dlogits, true));
  const BalPlan p = plan_balance(*shape, num_seqs);
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_LAUNCH(launch_balance_loss(*shape, p, workspace, coef->balance, coef->z, logits, topk_idx, seq_offsets,
                                 num_seqs, token_mask, loss, load, prob, dlogits, stream));
  return LC_MOE_OK;
}

lc_moe_status lc_moe_gate_backward(const lc_moe_shape* shape, const void* x, const void* ffn_rows,
                                   int32_t num_rows, const int32_t* slot_row, const void* dy, float* dgate,
                                   hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  if (num_rows < 0 || num_rows > shape->T * shape->K) return LC_MOE_E_SHAPE;
  LCM_CHECK(check_ptr(x));
  LCM_CHECK(check_ptr(ffn_rows, num_rows == 0));
  LCM_CHECK(check_ptr(slot_row));
  LCM_CHECK(check_ptr(dy));
  LCM_CHECK(check_ptr(dgate));
  LCM_LAUNCH(launch_gate_backward(*shape, x, ffn_rows, num_rows, slot_row, dy, dgate, stream));
  return LC_MOE_OK;
}

size_t lc_moe_router_backward_workspace_size(const lc_moe_shape* shape) {
  if (check_shape(shape) != LC_MOE_OK) return 0;
  return plan_router_backward(*shape).total;
}

lc_moe_status lc_moe_router_backward(const lc_moe_shape* shape, const void* x, const float* w_router,
                                     const float* logits, const int32_t* topk_idx, const float* dgate,
                                     const float* dlogits_aux, const void* dx_add, void* dx, float* dw_router,
                                     float* dlogits, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  LCM_CHECK(check_shape(shape));
  const RouterBwPlan p = plan_router_backward(*shape);
  LCM_CHECK(check_ptr(x, !dw_router));
  LCM_CHECK(check_ptr(w_router, !dx));
  LCM_CHECK(check_ptr(dgate, true));
  LCM_CHECK(check_ptr(logits, !dgate));
  LCM_CHECK(check_ptr(topk_idx, !dgate));
  LCM_CHECK(check_ptr(dlogits_aux, true));
  LCM_CHECK(check_ptr(dx_add, true));
  LCM_CHECK(check_ptr(dx, true));
  LCM_CHECK(check_ptr(dw_router, true));
  LCM_CHECK(check_ptr(dlogits, true));
  LCM_CHECK(check_space(workspace, workspace_bytes, p.total));
  LCM_LAUNCH(launch_router_backward(*shape, p, workspace, x, w_router, logits, topk_idx, dgate, dlogits_aux, dx_add,
                                    dx, dw_router, dlogits, stream));
  return LC_MOE_OK;
}

lc_moe_status lc_moe_adamw(const lc_moe_adamw_tensor* tensors, int32_t count, const lc_moe_adamw_hyper* hyper,
                           hipStream_t stream) {
  if (!hyper) return LC_MOE_E_NULLPTR;
  const lc_moe_adamw_hyper& h = *hyper;
  if (count < 0 || (h.state_bits != 8 && h.state_bits != 32)) return LC_MOE_E_SHAPE;
  if (!h.step_dev && h.step < 1) return LC_MOE_E_SHAPE;
  if (!(h.beta1 >= 0.f && h.beta1 < 1.f) || !(h.beta2 >= 0.f && h.beta2 < 1.f)) return LC_MOE_E_SHAPE;
  if (!(h.eps >= FLT_MIN || h.eps == 0.f)) return LC_MOE_E_SHAPE;  // (negative and NaN too)
  LCM_CHECK(check_ptr(h.step_dev, true));
  LCM_CHECK(check_ptr(h.grad_scale, true));
  if (count == 0) return LC_MOE_OK;
  if (!tensors) return LC_MOE_E_NULLPTR;
  for (int i = 0; i < count; ++i) {
    const lc_moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (int64_t(1) << 40)) return LC_MOE_E_SHAPE;
    if (t.param_dtype != LC_MOE_F32 && t.param_dtype != LC_MOE_BF16) return LC_MOE_E_DTYPE;
    if (t.grad_dtype != LC_MOE_F32 && t.grad_dtype != LC_MOE_BF16) return LC_MOE_E_DTYPE;
    if (t.n == 0) continue;
    LCM_CHECK(check_ptr(t.param));
    LCM_CHECK(check_ptr(t.master, true));
    LCM_CHECK(check_ptr(t.grad));
    LCM_CHECK(check_ptr(t.m));
    LCM_CHECK(check_ptr(t.v));
    LCM_CHECK(check_ptr(t.m_scale, h.state_bits == 32));
    LCM_CHECK(check_ptr(t.v_scale, h.state_bits == 32));
  }
  LCM_LAUNCH(launch_adamw(tensors, count, h, stream));
  return LC_MOE_OK;
}

}  // extern "C"
