// Internal definitions of the training operators (include/lc_moe_train.h).
#pragma once

#include "common.h"
#include "lc_moe_train.h"

namespace lcm {

// ---- balance loss --------------------------------------------------------------------
// Tokens per block of the statistics pass.  A block's tokens may belong to several
// sequences; its share of sequence s is partial row (block + s): along the tokens either
// the block or the sequence (or both) goes up from one share to the next, so these numbers
// are all different and below blocks + sequences.
constexpr int kBalTok = 64;

struct TokStat {  // what the gradient needs of a token's softmax
  float m, rs, lse;  // largest logit, 1 / sum of exponentials, m + log of that sum
  int32_t seq;       // the token's sequence; -1: the token does not count
};

struct BalPlan {
  size_t stat, part_p, part_c, part_n, part_z, seq_n, seq_z, seq_loss, factors, total;
  int nblocks, nparts, n_eb;  // token blocks, partial rows, blocks of 64 experts
};
inline BalPlan plan_balance(const lc_moe_shape& s, int S) {
  BalPlan p{};
  const size_t T = s.T, E = size_t(s.N) + s.Z;
  p.nblocks = int((T + kBalTok - 1) / kBalTok);
  p.nparts = p.nblocks + S;
  p.n_eb = int((E + 63) / 64);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  p.stat = take(T * sizeof(TokStat));
  p.part_p = take(size_t(p.nparts) * E * 4);
  p.part_c = take(size_t(p.nparts) * E * 4);
  p.part_n = take(size_t(p.nparts) * 4);
  p.part_z = take(size_t(p.nparts) * 4);
  p.seq_n = take(size_t(S) * 4);
  p.seq_z = take(size_t(S) * 4);
  p.seq_loss = take(size_t(S) * p.n_eb * 4);
  p.factors = take(8);
  p.total = o;
  return p;
}
hipError_t launch_balance_loss(const lc_moe_shape& s, const BalPlan& p, void* ws, float balance, float z,
                               const float* logits, const int32_t* idx, const int32_t* offsets, int S,
                               const uint8_t* mask, float* loss, int32_t* load, float* prob, float* dlogits,
                               hipStream_t st);

// ---- gate gradient -------------------------------------------------------------------
hipError_t launch_gate_backward(const lc_moe_shape& s, const void* x, const void* rows, int num_rows,
                                const int32_t* slot_row, const void* dy, float* dgate, hipStream_t st);

// ---- router backward -----------------------------------------------------------------
struct RouterBwPlan {
  size_t dl, total;
};
inline RouterBwPlan plan_router_backward(const lc_moe_shape& s) {
  RouterBwPlan p{};
  const size_t T = s.T, E = size_t(s.N) + s.Z;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  p.dl = take(T * E * 4);
  p.total = o;
  return p;
}
hipError_t launch_router_backward(const lc_moe_shape& s, const RouterBwPlan& p, void* ws, const void* x,
                                  const float* w_router, const float* logits, const int32_t* idx,
                                  const float* dgate, const float* aux, const void* dx_add, void* dx, float* dw,
                                  float* dlogits, hipStream_t st);

// ---- AdamW ---------------------------------------------------------------------------
hipError_t launch_adamw(const lc_moe_adamw_tensor* tensors, int count, const lc_moe_adamw_hyper& h, hipStream_t st);

}  // namespace lcm
