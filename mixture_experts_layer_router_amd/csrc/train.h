// Internal definitions of the training operators (include/lc_moe_train.h).
#pragma once

#include "common.h"
#include "lc_moe_train.h"

namespace lcm {

// ---- balance loss --------------------------------------------------------------------
// The statistics pass cuts the tokens into blocks.  A block's tokens may belong to several
// sequences; its share of sequence s is partial row (block + s): along the tokens either
// the block or the sequence (or both) goes up from one share to the next, so these numbers
// are all different and below blocks + sequences.
struct TokStat {  // what the gradient needs of a token's softmax
  float m, rs, lse;  // largest logit, 1 / sum of exponentials, m + log of that sum
  int32_t seq;       // the token's sequence; -1: the token does not count
};

struct BalPlan {
  size_t stat, part_p, part_c, part_n, part_z, seq_n, seq_z, seq_loss, total;
  int tok, nblocks, nparts, n_eb;  // tokens of a block, blocks, partial rows, runs of 64 experts
  bool one;                        // all in one workgroup
};
inline BalPlan plan_balance(const lc_moe_shape& s, int S) {
  BalPlan p{};
  const size_t T = s.T, E = size_t(s.N) + s.Z;
  // one block per CU until a block has 32 tokens (at least 4, a power of two)
  p.tok = 4;
  while (p.tok < 32 && size_t(p.tok) * 256 < T) p.tok *= 2;
  p.one = T <= 64 && T * E <= 16384 && S <= 2;
  if (p.one) p.tok = 64;
  p.nblocks = int((T + p.tok - 1) / p.tok);
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
// The two products run on the matrix cores, their fp32 operands cut into parts (router_grad.hip).
//   few    at most 64 tokens: dx straight from the fp32 weight
//   small  128 x 128 tiles, dlogits as bf16 parts, fp32 W_r and tokens cut in registers
//   big    bf16 layers: 128 x 256 tiles, dx from two scaled fp16 parts
// Ep: E rounded up to whole operand rows (32 experts).
enum RbForm { kRbFew, kRbSmall, kRbBig };
struct RouterBwPlan {
  size_t dl, dl16, rscale, wp, wexp, part, zero, total;
  int Ep;
  RbForm form;
  int splits, chunk;  // dW: pieces of the reduction over the tokens, tokens of each (x 32)
};
inline RouterBwPlan plan_router_backward(const lc_moe_shape& s) {
  RouterBwPlan p{};
  const size_t T = s.T, E = size_t(s.N) + s.Z;
  const bool bf = s.dtype == LC_MOE_BF16;
  p.Ep = int((E + 31) / 32 * 32);
  auto tiles = [](size_t m, size_t n, size_t bm, size_t bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
  // wide tiles where they fill the chip one and a half times (T = 8192, d = 6144, E = 128: 131 us
  // against 147 with the small ones; T = 2048, d = 6144, E = 768, 384 tiles: 154 against 184;
  // T = 4096, d = 2048, E = 96, 256 tiles: 43 against 34)
  const bool big = bf && T > 64 && tiles(T, s.d, 128, 256) >= 384;
  p.form = T <= 64 ? kRbFew : big ? kRbBig : kRbSmall;
  // dW: pieces for one workgroup a CU, beside dx's.  Wide tiles: of at least 512 tokens, and of at
  // most 4096 while that is for no more than four workgroups a CU, since a long piece ends behind
  // everything else (T = 2048, d = 6144, E = 768, one piece: 133 us against 154 for three; T = 4096,
  // E = 384, three: 142 against 160 for seven; T = 16384, E = 768, four: 0.946 ms against 0.990 for
  // one).  Small ones: of at least 128 (T = 4096, d = 2048, E = 96: 34 us against 36 for twice as many).
  const size_t t = tiles(E, s.d, 128, big ? 256 : 128), of4096 = (T + 4095) / 4096;
  size_t want = 256 / t;
  if (big && want < of4096) want = of4096 < 1024 / t ? of4096 : 1024 / t;
  const size_t least = big ? 512 : 128, most = (T + least - 1) / least;
  want = want > most ? most : want < 1 ? 1 : want;
  p.chunk = int((T + want - 1) / want + 31) / 32 * 32;
  p.splits = int((T + p.chunk - 1) / p.chunk);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
  p.dl = take(3 * T * p.Ep * 2);
  p.dl16 = take(big ? 2 * T * p.Ep * 2 : 0);
  p.rscale = take(big ? T * 4 : 0);
  p.wp = take(big ? 2 * size_t(p.Ep) * s.d * 2 : 0);
  p.wexp = take(big ? size_t(p.Ep) * 4 : 0);
  p.part = take(p.splits > 1 ? size_t(p.splits) * E * s.d * 4 : 0);
  p.zero = take(16);
  p.total = o;
  return p;
}
hipError_t launch_router_backward(const lc_moe_shape& s, const RouterBwPlan& p, void* ws, const void* x,
                                  const float* w_router, const float* logits, const int32_t* idx,
                                  const float* dgate, const float* aux, const void* dx_add, void* dx, float* dw,
                                  float* dlogits, hipStream_t st);

// Two values to bf16, nearest even, the first in the low half (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// ---- AdamW ---------------------------------------------------------------------------
hipError_t launch_adamw(const lc_moe_adamw_tensor* tensors, int count, const lc_moe_adamw_hyper& h, hipStream_t st);

}  // namespace lcm
