// Backward of the router: the softmax's gradient from the gates' gradients, then the two
// products with the router weight and with the tokens (formulas in
// include/lc_moe_train.h).
//
//   weight_f16_kernel  big layers of bf16 tokens: W_r as fp16, scaled row by row
//   operands_kernel    dlogits, one wave per token, cut into the products' operands
//   products_kernel    dx = dlogits W_r (+ dx_add) and dW = dlogits^T x on the matrix cores, side
//                      by side in one grid
//   sum_parts_kernel   the pieces of dW's reduction over the tokens, added in order
//
// What bounds it.  T = 16384, d = 6144, E = 768, bf16: 0.91 ms.  dW's three products of
// 155 GFLOP take 0.37-0.40 ms, 1.15-1.25 PFLOP/s, the rate of a large library product (1.2
// measured on this card); dx's three take 0.45 with 0.4 GB of dx_add and dx (one took 0.20-0.22);
// the operands 0.045, W_r 0.011, the sum of dW's four pieces 0.018.  One 155 GFLOP product
// each in fp32 (150 TFLOP/s) would take 1.0 ms.  Steps that got it there: 8.0 ms on plain fp32
// tiles, 0.95 on bf16 parts; dx from fp16 rows, of one part, 0.77, 0.71 with two workgroups a CU and
// dx through LDS, 0.65 with constant waits, dx_add loaded early and lane offsets kept; with the
// second part 0.97, 0.91 with both in one stage.
// Few tokens and narrow pools are bound by their launches and by a few memory latencies
// each: T = 64, d = 6144, E = 768 takes 22.1 us (operands 6, products 16), T = 4096, d = 2048,
// E = 96 takes 34 (6, 25, sum 4), fp32 T = 1777, d = 1028, E = 77 takes 20.
//
// Precision.  dW is an fp32 output: dlogits is cut into three bf16 parts (24 bits), the tokens
// are bf16 already (or cut the same way), every product of parts is exact and the matrix cores
// add them in fp32.  dx is made the same way.  That of a bf16 layer is rounded to bf16, but the
// rows of W_r may share a part that cancels in it (a row of the gates' dlogits sums to 0), so
// digits that its operands lose can show many times as large (two bf16 parts each, 16 bits, took
// 19.7 us at T = 64 and 31.1 at T = 4096).  The form for many tokens takes two fp16 parts of each
// operand, a power of two taken out of every row, and three products: an operand is off by at most
// 2^-23 of its value (2^-39 of its row's largest below 2^-17 of that), a product by 2^-21, less
// than its sums in fp32.  (One fp16 part of each, 11 bits, took 0.65 ms for the whole call; with
// rows of W_r that are ten parts shared to one part different, dx was off by 3.4e-3, where bf16's
// rounding alone is 1.7e-3.)
#include <type_traits>

#include "train.h"
#include "lanes.h"
#include "lds_dma.h"
#include "logit_row.h"

namespace lcm {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// v = h + m + l exactly but for the last of its 24 significant bits (each part keeps 8, the
// remainders are exact in fp32).
__device__ __forceinline__ void cut3(float v, bf16_t (&o)[3]) {
  o[0] = f2bf(v);
  const float r1 = v - bf2f(o[0]);
  o[1] = f2bf(r1);
  o[2] = f2bf(r1 - bf2f(o[1]));
}

// The same of 8 values, NP parts, as operands of the matrix cores.
template <int NP>
__device__ __forceinline__ void cut8(const float (&v)[8], bf16x8 (&o)[NP]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 u[NP];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
    for (int z = 0; z < NP; ++z) {
      const uint32_t w = pack_bf16(a, b);
      u[z][j] = w;
      a -= __uint_as_float(w << 16);
      b -= __uint_as_float(w & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int z = 0; z < NP; ++z) o[z] = __builtin_bit_cast(bf16x8, u[z]);
}

// v as the sum of two fp16 numbers, the value to nearest and what is left of it: off by 2^-23 of v
// (a unit of fp32's last place), or by 2^-25 where the second falls below fp16's normal numbers.
__device__ __forceinline__ void cut16(float v, bf16_t (&o)[2]) {
  const _Float16 h = static_cast<_Float16>(v);
  o[0] = __builtin_bit_cast(bf16_t, h);
  o[1] = __builtin_bit_cast(bf16_t, static_cast<_Float16>(v - static_cast<float>(h)));
}

// Exponent of the largest magnitude, so that 2^(14 - it) brings it into [2^14, 2^15), well inside
// fp16; -300 for a row of zeros, so that 2^it times any fp32 number is 0 and the scale of a token's
// row is taken from the experts whose W_r is not zero.
__device__ __forceinline__ int top_exp(float amax) { return amax > 0.f ? ilogbf(amax) : -300; }

// W_r row by row as two fp16 parts: the sum of w16[0][e] and w16[1][e] is 2^(14 - x) w[e], wexp[e]
// = x.  One workgroup per row; rows from E on are zeros.  [2][rows][d], a row per workgroup.
__global__ __launch_bounds__(256) void weight_f16_kernel(const float* __restrict__ w, bf16_t* __restrict__ w16,
                                                         int32_t* __restrict__ wexp, int E, int d) {
  __shared__ float wm[4];
  const int e = blockIdx.x, tid = threadIdx.x;
  const float* row = w + size_t(e) * d;
  float amax = 0.f;
  if (e < E) {
    for (int c = tid * 4; c < d; c += 1024) {
      const float4 q = *reinterpret_cast<const float4*>(row + c);
      amax = fmaxf(fmaxf(amax, fmaxf(fabsf(q.x), fabsf(q.y))), fmaxf(fabsf(q.z), fabsf(q.w)));
    }
  }
  amax = __ockl_wfred_max_f32(amax);
  if ((tid & 63) == 0) wm[tid >> 6] = amax;
  __syncthreads();
  const int x = top_exp(fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3])));
  if (tid == 0) wexp[e] = x;
  for (int c = tid * 4; c < d; c += 1024) {
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e < E) q = *reinterpret_cast<const float4*>(row + c);
    bf16_t h[4][2];
    cut16(ldexpf(q.x, 14 - x), h[0]), cut16(ldexpf(q.y, 14 - x), h[1]);
    cut16(ldexpf(q.z, 14 - x), h[2]), cut16(ldexpf(q.w, 14 - x), h[3]);
#pragma unroll
    for (int z = 0; z < 2; ++z)
      *reinterpret_cast<uint2*>(w16 + (size_t(z) * gridDim.x + e) * d + c) =
          make_uint2(h[0][z] | (uint32_t(h[1][z]) << 16), h[2][z] | (uint32_t(h[3][z]) << 16));
  }
}

struct OperandArgs {
  const float* logits;
  const int32_t* idx;
  const float* dgate;
  const float* aux;
  float* out;        // dlogits in fp32, or NULL
  bf16_t* parts;     // [3][T][Ep]
  bf16_t* dl16;      // [2][T][Ep] fp16 parts of 2^(wexp[e] + 14 - x) dlogits, x the row's exponent;
                     // or NULL
  float* rscale;     // [T] 2^(x - 28)
  const int32_t* wexp;
  int T, E, K, Ep;
  uint4* zero;       // 16 zero bytes: the source of operand chunks past the data
};

// dlogits of four tokens, one per wave, the row in its registers as in logit_row.h; the picks'
// gradients are added in pick order by the lane that holds the expert.
template <int EPL, int V>
__global__ __launch_bounds__(256) void operands_kernel(OperandArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.zero = make_uint4(0, 0, 0, 0);
  constexpr int J = EPL / V;  // runs of 64 V experts
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int E = a.E, K = a.K;
  if (t >= a.T) return;
  float v[EPL], ax[EPL];
  if (a.dgate) load_row<EPL, V>(a.logits + size_t(t) * E, E, lane, -INFINITY, v);
  if (a.aux) load_row<EPL, V>(a.aux + size_t(t) * E, E, lane, 0.f, ax);
  if (a.dgate) {
    const RowSum r = softmax_row<EPL>(v);
    const float rs = r.m > -INFINITY ? 1.f / r.sum : 0.f;
    float dp[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) dp[i] = 0.f;
    for (int k0 = 0; k0 < K; k0 += 64) {
      const int n = K - k0 < 64 ? K - k0 : 64;
      int pe = -1;
      float pg = 0.f;
      if (lane < n) {
        pe = a.idx[size_t(t) * K + k0 + lane];
        pg = a.dgate[size_t(t) * K + k0 + lane];
      }
      for (int k = 0; k < n; ++k) {
        const int e = __builtin_amdgcn_readlane(pe, k);
        const float g = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, pg), k));
        if (unsigned(e) >= unsigned(E)) continue;
        const bool mine = ((e / V) & 63) == lane;
        const int jk = e / (64 * V), c = e % V;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j != jk) continue;
#pragma unroll
          for (int w = 0; w < V; ++w) dp[j * V + w] += mine && w == c ? g : 0.f;
        }
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] *= rs;
      dot += v[i] * dp[i];
    }
    dot = __ockl_wfred_add_f32(dot);
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] *= dp[i] - dot;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = 0.f;
  }
  if (a.aux) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] += ax[i];
  }
  if (a.out) store_row<EPL, V>(a.out + size_t(t) * E, E, lane, v);
  auto put = [&](bf16_t* dst, int j, const bf16_t (&h)[V]) {
    const int e = (j * 64 + lane) * V;
    if (e >= a.Ep) return;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst + e) = make_uint2(h[0] | (uint32_t(h[1]) << 16), h[2] | (uint32_t(h[3]) << 16));
    else
      dst[e] = h[0];
  };
  const size_t plane = size_t(a.T) * a.Ep;
  bf16_t* row = a.parts + size_t(t) * a.Ep;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    bf16_t h[3][V];
#pragma unroll
    for (int w = 0; w < V; ++w) {
      bf16_t c[3];
      cut3((j * 64 + lane) * V < E ? v[j * V + w] : 0.f, c);
      h[0][w] = c[0], h[1][w] = c[1], h[2][w] = c[2];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) put(row + q * plane, j, h[q]);
  }
  if (a.dl16) {
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int w = 0; w < V; ++w) {
        const int e = (j * 64 + lane) * V + w;
        v[j * V + w] = e < E ? ldexpf(v[j * V + w], a.wexp[e]) : 0.f;
        amax = fmaxf(amax, fabsf(v[j * V + w]));
      }
    int x = top_exp(__ockl_wfred_max_f32(amax));
    x = x < -98 ? -98 : x;  // 2^(x - 28) is a normal fp32 number
#pragma unroll
    for (int j = 0; j < J; ++j) {
      bf16_t h[2][V];
#pragma unroll
      for (int w = 0; w < V; ++w) {
        bf16_t c[2];
        cut16(ldexpf(v[j * V + w], 14 - x), c);
        h[0][w] = c[0], h[1][w] = c[1];
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) put(a.dl16 + q * plane + size_t(t) * a.Ep, j, h[q]);
    }
    if (lane == 0) a.rscale[t] = ldexpf(1.f, x - 28);
  }
}

// ---------------------------------------------------------------------------------------
// One tile of C[M][N] = sum over pairs of parts (a, b) of A_a B_b, fp32 accumulation on
// v_mfma_f32_32x32x16.  A stage holds BK reduction steps of NA parts of A and NB parts of B, so
// a loaded part serves every product it takes part in: with the pairs a + b < max(NA, NB)
// (h x, m x, l x of three and one; h h, h m, m h of two each; the six largest of three and three)
// the operand tiles of a stage carry 3 or 6 products.
//   DX: A(m, k) = dlogits, row m, K-contiguous; B(k, n) = W_r, row k.
//   DW: A(m, k) = dlogits, row k (a token), M-contiguous; B(k, n) = tokens, row k.
// F16: A and B are two fp16 parts each; the product of two low parts, left out, is 2^-22 of the
// whole.  A stage of 16 steps with both parts of both reads 94 bytes of LDS a clock at the matrix
// cores' full rate; the three products one after another, 32 steps of one part of each a stage,
// would need 140, more than the 128 there are (0.91 ms against 0.97 for the call).
// CUT: B is fp32 (W_r; fp32 tokens) and lies in LDS as such; a wave cuts its fragments into the
// NB parts in registers.  (Parts cut by a launch before take 6 bytes a value, so 96 KB of LDS and
// one workgroup a CU, and a pass over x and W_r: fp32 T = 4096, d = 2048, E = 96 took 69 us, now 51;
// T = 4096, d = 2800, E = 384 184, now 144.)
// Tile BM x BN, 64 x (BN / 2) outputs per wave, BM / 32 waves, a ring of NST stages in LDS
// filled by direct global->LDS loads.  Operands whose output index is contiguous lie in LDS
// as in memory ([BK][columns]) and are read by the transposing LDS read; 16-byte chunk c of
// row r sits in the 32-byte granule (c / 2) ^ 2 (r % 4), which spreads the four rows of a
// read over the banks; fp32 chunk c of row r sits in c ^ 8 (r / 8 % 2), so that the two halves of
// a wave, 8 rows apart, read different banks.  K-contiguous rows are 64 bytes, chunk c in slot
// c ^ swz4(r), or 32 bytes, c ^ (r / 4 % 2).
// ---------------------------------------------------------------------------------------
struct ProdArgs {
  const bf16_t* a;  // [NA][T][Ep]
  const void* b;    // DX: [krows][ldb] (F16: [2][krows][ldb]); DW: [T][ldb]
  size_t plane_a;
  const bf16_t* zero;
  const void* add;
  void* c;
  const float* rscale;  // fp16: units of the rows' sums
  int M, N, Kdim, lda, ldb;
  int krows;            // rows of B: the reduction's steps behind them have zeros in A
  int chunk;            // reduction steps of a piece (a multiple of 32)
  int n_mt, n_nt, splits;
};

template <bool DX, bool F16, bool CUT, int BM, int BN, int NA, int NB, int BK, int NST, typename Tc>
__device__ __forceinline__ void product_tile(const ProdArgs& p, unsigned block, unsigned char* smem) {
  constexpr int WAVES = BM / 32, WN = 2, WC = BN / WN;  // wave tile: 64 x WC
  constexpr int NBL = WC / 32;                          // 32-wide column blocks of a wave
  constexpr int EB = CUT ? 4 : 2, CC = 16 / EB;            // bytes of an element of B, columns of a chunk
  constexpr int A_OP = BM * BK * 2, B_OP = BN * BK * EB;  // bytes of A's parts (each) and of B in a stage
  constexpr int NL = CUT ? 1 : NB;                        // parts of B that are loaded
  constexpr int STAGE = NA * A_OP + NL * B_OP;
  constexpr int NP = NA > NB ? NA : NB;
  constexpr int LA = A_OP / 1024 / WAVES, LB = B_OP / 1024 / WAVES;  // direct loads of a wave
  constexpr int LOADS = NA * LA + NL * LB;                           // and per stage
  static_assert(A_OP % (1024 * WAVES) == 0 && B_OP % (1024 * WAVES) == 0, "whole loads");
  static_assert(!DX || BK == 32 || BK == 16, "K-contiguous rows are staged 64 or 32 bytes at a time");
  static_assert(NBL == 2 || NBL == 4, "wave tiles of 64 or 128 columns");

  // unit: pieces of the reduction, in them groups of 8 M-tiles, in a group column tiles, in them
  // its M-tiles; each XCD takes a contiguous eighth, so workgroups side by side share operand
  // rows in its L2
  const int U = p.n_mt * p.n_nt * p.splits, per = (U + 7) >> 3, slot_w = block >> 3;
  if (slot_w >= per) return;
  const int u = (block & 7) * per + slot_w;
  if (u >= U) return;
  const int tiles = p.n_mt * p.n_nt, sp = u / tiles;
  int r0 = u - sp * tiles;
  const int grp = r0 / (8 * p.n_nt);
  r0 -= grp * 8 * p.n_nt;
  const int gm = p.n_mt - grp * 8 < 8 ? p.n_mt - grp * 8 : 8;
  const int m0 = (grp * 8 + r0 % gm) * BM, n0 = (r0 / gm) * BN;
  const int kbeg = sp * p.chunk, kend = kbeg + p.chunk < p.Kdim ? kbeg + p.chunk : p.Kdim;
  const int nk = (kend - kbeg + BK - 1) / BK;
  const int krows = kend < p.krows ? kend : p.krows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // A wave's load i of an operand with contiguous columns (BC of 2 bytes) fills bytes
  // 1024 (wave + WAVES i) of its part: 512 / BC rows of 2 BC bytes.
  auto col_place = [&](int BC, int i, int& kr, int& ch) {  // the lane's row and 16-byte chunk
    const int rpl = 512 / BC, cpr = BC / 8;  // rows of a load, chunks of a row
    const int sl = lane % cpr;
    kr = rpl * (wave + WAVES * i) + lane / cpr;
    ch = 2 * ((sl >> 1) ^ (2 * (kr & 3))) + (sl & 1);
  };
  auto b_place = [&](int i, int& kr, int& ch) {
    if constexpr (CUT) {
      constexpr int RPL = 256 / BN, CPR = BN / 4;
      kr = RPL * (wave + WAVES * i) + lane / CPR;
      ch = (lane % CPR) ^ (8 * (kr >> 3 & 1));
    } else {
      col_place(BN, i, kr, ch);
    }
  };
  // Whole stages: the lane's byte offset from the stage's first element does not change, so a
  // load is a scalar base and that offset.  Columns past the operand repeat a valid column and
  // rows past M a valid row; neither is stored.
  auto swz = [](int r) { return BK == 32 ? swz4(r) : r >> 2 & 1; };  // K-contiguous row r
  uint32_t off_a[LA], off_b[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    if constexpr (DX) {
      constexpr int CPR = BK / 8;  // chunks of a row
      const int r = 64 / CPR * (wave + WAVES * i) + lane / CPR;
      off_a[i] = uint32_t(m0 + r < p.M ? r : 0) * p.lda * 2 + ((lane % CPR) ^ swz(r)) * 16;
    } else {
      int kr, ch;
      col_place(BM, i, kr, ch);
      off_a[i] = uint32_t(kr) * p.lda * 2 + (m0 + ch * 8 < p.lda ? ch * 16 : 0);
    }
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    int kr, ch;
    b_place(i, kr, ch);
    off_b[i] = uint32_t(kr) * p.ldb * EB + (n0 + ch * CC < p.ldb ? ch * 16 : 0);
  }
  const bool near = p.ldb < (1 << 24);  // 32 rows within 2^32 bytes
  auto issue = [&](int kt) {
    unsigned char* st = smem + (kt % NST) * STAGE;
    unsigned char* sb = st + NA * A_OP;
    const int k0 = kbeg + kt * BK;
    const bf16_t* a0 = DX ? p.a + size_t(m0) * p.lda + k0 : p.a + size_t(k0) * p.lda + m0;
    const char* b0 = static_cast<const char*>(p.b) + (size_t(k0) * p.ldb + n0) * EB;
    const size_t plane_b = size_t(p.krows) * p.ldb * EB;  // bytes of a part of B
    if (near && k0 + BK <= krows) {
#pragma unroll
      for (int q = 0; q < NA; ++q) {
        const char* g = reinterpret_cast<const char*>(a0 + q * p.plane_a);
#pragma unroll
        for (int i = 0; i < LA; ++i) dma16(g + off_a[i], st + q * A_OP + (wave + WAVES * i) * 1024);
      }
#pragma unroll
      for (int q = 0; q < NL; ++q)
#pragma unroll
        for (int i = 0; i < LB; ++i) dma16(b0 + q * plane_b + off_b[i], sb + q * B_OP + (wave + WAVES * i) * 1024);
      return;
    }
    // a piece's last, partial stage: rows past its end (the tokens of dW, W_r's last) are zeros
    for (int q = 0; q < NA; ++q)
      for (int i = 0; i < LA; ++i) {
        const bf16_t* g;
        if constexpr (DX) {
          g = reinterpret_cast<const bf16_t*>(reinterpret_cast<const char*>(a0 + q * p.plane_a) + off_a[i]);
        } else {
          int kr, ch;
          col_place(BM, i, kr, ch);
          const bool in = k0 + kr < kend && m0 + ch * 8 < p.lda;
          g = in ? a0 + q * p.plane_a + size_t(kr) * p.lda + ch * 8 : p.zero;
        }
        dma16(g, st + q * A_OP + (wave + WAVES * i) * 1024);
      }
    for (int q = 0; q < NL; ++q)
      for (int i = 0; i < LB; ++i) {
        int kr, ch;
        b_place(i, kr, ch);
        const bool in = k0 + kr < krows && n0 + ch * CC < p.ldb;
        dma16(in ? b0 + q * plane_b + size_t(kr) * p.ldb * EB + ch * 16 : reinterpret_cast<const char*>(p.zero),
              sb + q * B_OP + (wave + WAVES * i) * 1024);
      }
  };

  const int l32 = lane & 31, khalf = lane >> 5;
  const int tr_j = (lane >> 2) & 3, tr_row = 8 * khalf + tr_j, tr_g = (lane >> 4) & 1, tr_byte = 8 * (lane & 3);
  typedef __attribute__((address_space(3))) unsigned char lds_u8;
  // LDS address of this lane's first row (of two, 4 apart) of the 32 columns at `base`
  auto tr_addr = [&](const unsigned char* op, int pitch, int base, int ks) -> uint32_t {
    const int lg = (base >> 4) + tr_g;
    const unsigned char* q = op + (ks + tr_row) * pitch + ((lg ^ (2 * tr_j)) << 5) + tr_byte;
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(reinterpret_cast<const lds_u8*>(
        reinterpret_cast<uintptr_t>(q))));
  };
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));

  f32x16 acc[2][NBL];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NBL; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  // bf16: dx_add of the wave's first 32 rows, loaded beside the stages (see the end)
  constexpr bool HALF = sizeof(Tc) == 2;
  constexpr int LPR = WC / 8, RPI = 64 / LPR, NG = HALF ? 32 / RPI : 1;  // lanes of a row, rows at a time
  const Tc* add = static_cast<const Tc*>(p.add);
  const int rl = lane / LPR, cl = (lane % LPR) * 8;
  uint4 q0[NG];
  auto load_add = [&](int i, uint4 (&q)[NG]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int m = m0 + wm * 64 + i * 32 + g * RPI + rl, n = n0 + wn * WC + cl;
      q[g] = add && m < p.M && n < p.N ? *reinterpret_cast<const uint4*>(add + size_t(m) * p.N + n) : make_uint4(0, 0, 0, 0);
    }
  };
  if constexpr (HALF) load_add(0, q0);
  const int npro = nk < NST ? nk : NST;
  for (int s = 0; s < npro; ++s) issue(s);

  for (int kt = 0; kt < nk; ++kt) {
    // stage kt landed: later stages up to kt + NST - 2 (at the start kt + NST - 1) are on their way
    // (a constant count but at both ends: the run-time count is a jump through a table)
    if (kt > 0 && kt + NST - 2 < nk) {
      LCM_WAIT_VMCNT((NST - 2) * LOADS);
    } else {
      const int last = kt + NST - 1 < nk ? kt + NST - 1 : nk - 1;
      wait_vmcnt((last - kt) * LOADS);
    }
    wait_lds_reads();
    block_barrier();  // every wave's loads of stage kt visible; stage kt - 1 read by all
    if (kt > 0 && kt + NST - 1 < nk) issue(kt + NST - 1);  // into stage kt - 1's slot
    const unsigned char* st = smem + (kt % NST) * STAGE;
    const unsigned char* sb = st + NA * A_OP;
    float bv[CUT ? BK / 16 : 1][NBL][8];  // the stage's fp32 values, read before any is waited for
    if constexpr (CUT) {
#pragma unroll
      for (int ks = 0; ks < BK; ks += 16)
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          const int c = wn * WC + 32 * j + l32;
          const float* f = reinterpret_cast<const float*>(sb + (ks + 8 * khalf) * (BN * 4) + (((c >> 2) ^ (8 * khalf)) << 4)) + (c & 3);
#pragma unroll
          for (int q = 0; q < 8; ++q) bv[ks / 16][j][q] = f[q * BN];
        }
    }
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      bf16x8 fa[NA][2], fb[NB][NBL];
      if constexpr (DX) {
#pragma unroll
        for (int q = 0; q < NA; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            fa[q][i] = *reinterpret_cast<const bf16x8*>(st + q * A_OP + (wm * 64 + i * 32 + l32) * (2 * BK) +
                                                        (((ks / 8 + khalf) ^ swz(l32)) << 4));
      }
      // Each block of transposing reads waits for itself (see ffn_wgrad_kernel).
      auto tr4 = [&](auto pitch, uint32_t a0, uint32_t a1, bf16x8& f0, bf16x8& f1) {
        constexpr int P = decltype(pitch)::value;
        uint64_t r[4];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4\n"
            "ds_read_b64_tr_b16 %1, %4 offset:%6\n"
            "ds_read_b64_tr_b16 %2, %5\n"
            "ds_read_b64_tr_b16 %3, %5 offset:%6\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
            : "v"(a0), "v"(a1), "n"(4 * P)
            : "memory");
        f0 = __builtin_bit_cast(bf16x8, u64x2{r[0], r[1]});
        f1 = __builtin_bit_cast(bf16x8, u64x2{r[2], r[3]});
      };
      auto tr8 = [&](auto pitch, const uint32_t (&ad)[4], bf16x8* f) {
        constexpr int P = decltype(pitch)::value;
        uint64_t r[8];
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8\n"
            "ds_read_b64_tr_b16 %1, %8 offset:%12\n"
            "ds_read_b64_tr_b16 %2, %9\n"
            "ds_read_b64_tr_b16 %3, %9 offset:%12\n"
            "ds_read_b64_tr_b16 %4, %10\n"
            "ds_read_b64_tr_b16 %5, %10 offset:%12\n"
            "ds_read_b64_tr_b16 %6, %11\n"
            "ds_read_b64_tr_b16 %7, %11 offset:%12\n"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
            : "v"(ad[0]), "v"(ad[1]), "v"(ad[2]), "v"(ad[3]), "n"(4 * P)
            : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __builtin_bit_cast(bf16x8, u64x2{r[2 * j], r[2 * j + 1]});
      };
      if constexpr (!DX) {
#pragma unroll
        for (int q = 0; q < NA; ++q)
          tr4(std::integral_constant<int, BM * 2>{}, tr_addr(st + q * A_OP, BM * 2, wm * 64, ks),
              tr_addr(st + q * A_OP, BM * 2, wm * 64 + 32, ks), fa[q][0], fa[q][1]);
      }
      if constexpr (CUT) {
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          bf16x8 h[NB];
          cut8<NB>(bv[ks / 16][j], h);
#pragma unroll
          for (int q = 0; q < NB; ++q) fb[q][j] = h[q];
        }
      } else if constexpr (NBL == 4) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
          uint32_t ad[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) ad[j] = tr_addr(sb + q * B_OP, BN * 2, wn * WC + 32 * j, ks);
          tr8(std::integral_constant<int, BN * 2>{}, ad, fb[q]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < NB; ++q)
          tr4(std::integral_constant<int, BN * 2>{}, tr_addr(sb + q * B_OP, BN * 2, wn * WC, ks),
              tr_addr(sb + q * B_OP, BN * 2, wn * WC + 32, ks), fb[q][0], fb[q][1]);
      }
#pragma unroll
      for (int qa = 0; qa < NA; ++qa)
#pragma unroll
        for (int qb = 0; qb < NB; ++qb) {
          if (qa + qb >= NP) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NBL; ++j) {
              if constexpr (F16)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, fa[qa][i]),
                                                                  __builtin_bit_cast(f16x8, fb[qb][j]), acc[i][j], 0, 0, 0);
              else
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[qa][i], fb[qb][j], acc[i][j], 0, 0, 0);
            }
        }
    }
  }

  // 32x32 D layout: column lane % 32, rows 8 (r / 4) + 4 (lane / 32) + r % 4
  if constexpr (HALF) {
    // bf16: 32 rows at a time through the wave's own piece of the ring, so that dx_add is read and
    // dx written 16 bytes a lane in whole lines (8 bytes a lane from the accumulators as they
    // lie took 120 us for dx_add and 60 us for dx at T = 16384, d = 6144)
    constexpr int PITCH = WC + 4;
    static_assert(WAVES * 32 * PITCH * 4 <= NST * STAGE, "fits the ring");
    Tc* out = static_cast<Tc*>(p.c);
    float* buf = reinterpret_cast<float*>(smem) + wave * 32 * PITCH;
    const int n = n0 + wn * WC + cl;
    uint4 q1[NG];
    load_add(1, q1);
    wait_lds_reads();
    block_barrier();  // the ring is read by all
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4(&q)[NG] = i == 0 ? q0 : q1;
      float un[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int m = m0 + wm * 64 + i * 32 + g * RPI + rl;
        un[g] = F16 && m < p.M ? p.rscale[m] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < NBL; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) buf[(8 * (r >> 2) + 4 * khalf + (r & 3)) * PITCH + j * 32 + l32] = acc[i][j][r];
      wait_lds_reads();  // (its writes: the same counter)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int m = m0 + wm * 64 + i * 32 + g * RPI + rl;
        const float* v = buf + (g * RPI + rl) * PITCH + cl;
        const float4 lo = *reinterpret_cast<const float4*>(v), hi = *reinterpret_cast<const float4*>(v + 4);
        const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const uint32_t u[4] = {q[g].x, q[g].y, q[g].z, q[g].w};
        uint32_t o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o[c] = f2bf(fmaf(w[2 * c], un[g], __uint_as_float(u[c] << 16))) |
                 (uint32_t(f2bf(fmaf(w[2 * c + 1], un[g], __uint_as_float(u[c] & 0xFFFF0000u)))) << 16);
        if (m < p.M && n < p.N) *reinterpret_cast<uint4*>(out + size_t(m) * p.N + n) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      wait_lds_reads();  // read before the next 32 rows are written
    }
  } else {
    // fp32: a transpose among four lanes gives each lane one row of 4 columns, 16 bytes
    const int q4 = lane & 3;
    float* out = static_cast<float*>(p.c) + (DX ? 0 : size_t(sp) * p.M * p.N);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NBL; ++j)
#pragma unroll
        for (int rq = 0; rq < 4; ++rq) {
          float v[4], w[4];
#pragma unroll
          for (int t4 = 0; t4 < 4; ++t4) v[t4] = acc[i][j][rq * 4 + t4];
          quad_transpose(v, q4, w);
          const int m = m0 + wm * 64 + i * 32 + 8 * rq + 4 * khalf + q4, n = n0 + wn * WC + j * 32 + (lane & 28);
          if (m >= p.M || n >= p.N) continue;
          const size_t o = size_t(m) * p.N + n;
          if (add) {
            const float4 q = *reinterpret_cast<const float4*>(add + o);
            w[0] += q.x, w[1] += q.y, w[2] += q.z, w[3] += q.w;
          }
          *reinterpret_cast<float4*>(out + o) = make_float4(w[0], w[1], w[2], w[3]);
        }
  }
}

// dx of at most 64 tokens: 32 columns a workgroup, every fourth 16-step of the reduction a
// wave, the four sums added through LDS in wave order (T = 64, d = 6144, E = 768: 22.1 us for the
// call).  W_r is read as it lies, once, and cut into NP parts in registers: lane (l32, half) holds
// column n0 + l32 of rows 8 half + 0..7.
template <int NP, typename Tx>
__device__ __forceinline__ void dx_few(const ProdArgs& p, const float* __restrict__ w, int E, unsigned block, float* sums) {
  const int n0 = block * 32;
  if (n0 >= p.N) return;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = n0 + l32 < p.N ? n0 + l32 : n0;
  // dx_add of the thread's 16 bytes of output (two of them for fp32), loaded beside the products:
  // it may be dx itself, so behind them each piece would wait for the last one's store
  constexpr int CH = 16 / sizeof(Tx), PIECES = 64 * 32 / CH / 256;
  const Tx* add = static_cast<const Tx*>(p.add);
  Tx* out = static_cast<Tx*>(p.c);
  uint4 q[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = i * 256 + tid, m = at / (32 / CH), c = n0 + at % (32 / CH) * CH;
    q[i] = add && m < p.M && c < p.N ? *reinterpret_cast<const uint4*>(add + size_t(m) * p.N + c) : make_uint4(0, 0, 0, 0);
  }
  const bf16_t* arow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = i * 32 + l32 < p.M ? i * 32 + l32 : 0;
    arow[i] = p.a + size_t(m) * p.lda + 8 * half;
  }
  f32x16 acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  // steps whose loads are in flight together (T = 64, E = 768: 22.1 us; four 22.2, six 24.2)
  constexpr int B = 3;
  float wv[B][8];
  bf16x8 fa[B][NP][2];
  auto load = [&](int b, int k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = k + 8 * half + j;
      wv[b][j] = w[size_t(e < E ? e : E - 1) * p.N + n];  // dlogits' columns past E are zero
    }
#pragma unroll
    for (int z = 0; z < NP; ++z)
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[b][z][i] = *reinterpret_cast<const bf16x8*>(arow[i] + z * p.plane_a + k);
  };
#pragma unroll
  for (int b = 0; b < B; ++b)
    if (wave * 16 + 64 * b < p.Kdim) load(b, wave * 16 + 64 * b);
  for (int k0 = wave * 16; k0 < p.Kdim; k0 += 64 * B) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (k0 + 64 * b >= p.Kdim) break;
      bf16x8 h[NP];
      cut8<NP>(wv[b], h);
#pragma unroll
      for (int qa = 0; qa < NP; ++qa)
#pragma unroll
        for (int qb = 0; qb + qa < NP; ++qb)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[b][qa][i], h[qb], acc[i], 0, 0, 0);
      if (k0 + 64 * (b + B) < p.Kdim) load(b, k0 + 64 * (b + B));
    }
  }
  float(*s)[64][33] = reinterpret_cast<float(*)[64][33]>(sums);  // [4][64 rows][32 columns + 1]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[wave][i * 32 + 8 * (r >> 2) + 4 * half + (r & 3)][l32] = acc[i][r];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = i * 256 + tid, m = at / (32 / CH), c = at % (32 / CH) * CH;
    if (m >= p.M || n0 + c >= p.N) continue;
    const uint32_t u[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
    float v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      v[j] = (s[0][m][c + j] + s[1][m][c + j]) + (s[2][m][c + j] + s[3][m][c + j]);
      if constexpr (sizeof(Tx) == 2) v[j] += __uint_as_float(j & 1 ? u[j >> 1] & 0xFFFF0000u : u[j >> 1] << 16);
      else v[j] += __uint_as_float(u[j]);
    }
    Tx* o = out + size_t(m) * p.N + n0 + c;
    if constexpr (sizeof(Tx) == 2) {
      uint32_t w2[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w2[j] = f2bf(v[2 * j]) | (uint32_t(f2bf(v[2 * j + 1])) << 16);
      *reinterpret_cast<uint4*>(o) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    } else {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Both products in one grid: dW's workgroups first (their tiles are the longest), then dx's.
// (Mixed one to three, so that both kinds share a CU, they took 1.6 ms instead of 0.64 at
// T = 16384, d = 6144, E = 768: their operands push each other out of the L2.)
struct ProductsArgs {
  ProdArgs dw, dx;
  unsigned dw_blocks;  // a multiple of 8
  const float* w;      // the fp32 weight (few tokens)
  int E;
};

template <int FORM, bool BF>
__global__ __launch_bounds__(256, 2) void products_kernel(ProductsArgs a) {
  typedef typename std::conditional<BF, bf16_t, float>::type Tx;
  constexpr int X = BF ? 1 : 3, W = 3;  // parts of the tokens; of W_r (and dlogits for dx)
  // ring: big 2 x 40 KB for dW, 3 x 24 KB for dx (16 steps each); else 2 x 40 KB (few bf16 tokens
  // 2 x 32 KB)
  constexpr int LDS = FORM == kRbFew && BF ? 65536 : 81920;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[LDS];
  if (blockIdx.x < a.dw_blocks) {
    if constexpr (FORM == kRbBig) product_tile<false, false, false, 128, 256, 3, 1, 32, 2, float>(a.dw, blockIdx.x, smem);
    else product_tile<false, false, !BF, 128, 128, 3, X, 32, 2, float>(a.dw, blockIdx.x, smem);
  } else {
    const unsigned b = blockIdx.x - a.dw_blocks;
    if constexpr (FORM == kRbFew) dx_few<W, Tx>(a.dx, a.w, a.E, b, reinterpret_cast<float*>(smem));
    else if constexpr (FORM == kRbSmall) product_tile<true, false, true, 128, 128, W, W, 32, 2, Tx>(a.dx, b, smem);
    else product_tile<true, true, false, 128, 256, 2, 2, 16, 3, Tx>(a.dx, b, smem);
  }
}

// dW = its pieces, added in order (n values, a multiple of 4; 4 per thread).
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                        int splits, size_t n) {
  const size_t i = (size_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float4 a = *reinterpret_cast<const float4*>(part + i);
  for (int s0 = 1; s0 < splits; s0 += 8) {
    float4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j < splits) b[j] = *reinterpret_cast<const float4*>(part + (s0 + j) * n + i);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j < splits) a.x += b[j].x, a.y += b[j].y, a.z += b[j].z, a.w += b[j].w;
  }
  *reinterpret_cast<float4*>(out + i) = a;
}

template <int FORM, bool BF>
static void launch_products(ProductsArgs a, hipStream_t st) {
  constexpr int BM = 128, BN = FORM == kRbBig ? 256 : 128;
  size_t dx_blocks = 0;
  if (a.dw.c) {
    a.dw.n_mt = (a.dw.M + BM - 1) / BM;
    a.dw.n_nt = (a.dw.N + BN - 1) / BN;
    a.dw_blocks = unsigned((size_t(a.dw.n_mt) * a.dw.n_nt * a.dw.splits + 7) / 8 * 8);
  }
  if (a.dx.c) {
    a.dx.n_mt = (a.dx.M + BM - 1) / BM;
    a.dx.n_nt = (a.dx.N + BN - 1) / BN;
    dx_blocks = FORM == kRbFew ? size_t(a.dx.N + 31) / 32 : (size_t(a.dx.n_mt) * a.dx.n_nt + 7) / 8 * 8;
  }
  hipLaunchKernelGGL((products_kernel<FORM, BF>), dim3(unsigned(a.dw_blocks + dx_blocks)), dim3(BM * 2), 0, st, a);
}

hipError_t launch_router_backward(const lc_moe_shape& s, const RouterBwPlan& p, void* ws, const void* x,
                                  const float* w_router, const float* logits, const int32_t* idx,
                                  const float* dgate, const float* aux, const void* dx_add, void* dx, float* dw,
                                  float* dlogits, hipStream_t st) {
  const int E = s.N + s.Z, epl = (E + 63) / 64;
  const bool bf = s.dtype == LC_MOE_BF16, f16 = p.form == kRbBig;
  char* w = static_cast<char*>(ws);
  bf16_t* wp = reinterpret_cast<bf16_t*>(w + p.wp);
  OperandArgs o{};
  o.logits = logits;
  o.idx = idx;
  o.dgate = dgate;
  o.aux = aux;
  o.out = dlogits;
  o.parts = reinterpret_cast<bf16_t*>(w + p.dl);
  o.zero = reinterpret_cast<uint4*>(w + p.zero);
  o.T = s.T;
  o.E = E;
  o.K = s.K;
  o.Ep = p.Ep;
  if (dx && f16) {
    o.dl16 = reinterpret_cast<bf16_t*>(w + p.dl16);
    o.rscale = reinterpret_cast<float*>(w + p.rscale);
    int32_t* wexp = reinterpret_cast<int32_t*>(w + p.wexp);
    o.wexp = wexp;
    hipLaunchKernelGGL(weight_f16_kernel, dim3(p.Ep), dim3(256), 0, st, w_router, wp, wexp, E, s.d);
  }
  const dim3 grid(unsigned((s.T + 3) / 4));
#define LCM_DL(n, v) hipLaunchKernelGGL((operands_kernel<n, v>), grid, dim3(256), 0, st, o)
  if (E % 4 == 0) {
    if (epl <= 4) LCM_DL(4, 4);
    else if (epl <= 8) LCM_DL(8, 4);
    else if (epl <= 12) LCM_DL(12, 4);
    else if (epl <= 16) LCM_DL(16, 4);
    else if (epl <= 32) LCM_DL(32, 4);
    else LCM_DL(64, 4);
  } else {
    if (epl <= 2) LCM_DL(2, 1);
    else if (epl <= 8) LCM_DL(8, 1);
    else if (epl <= 16) LCM_DL(16, 1);
    else if (epl <= 32) LCM_DL(32, 1);
    else LCM_DL(64, 1);
  }
#undef LCM_DL
  if (!dx && !dw) return hipGetLastError();
  ProductsArgs a{};
  a.w = w_router;
  a.E = E;
  ProdArgs q{};
  q.lda = p.Ep;
  q.ldb = s.d;
  q.zero = reinterpret_cast<const bf16_t*>(o.zero);
  q.N = s.d;
  a.dx = a.dw = q;
  a.dx.a = f16 ? o.dl16 : o.parts;
  a.dx.plane_a = size_t(s.T) * p.Ep;
  a.dx.b = f16 ? static_cast<const void*>(wp) : w_router;
  a.dx.krows = f16 ? p.Ep : E;
  a.dx.rscale = o.rscale;
  a.dx.M = s.T;
  a.dx.Kdim = a.dx.chunk = p.Ep;
  a.dx.splits = 1;
  a.dx.add = dx_add;
  a.dx.c = dx;
  a.dw.a = o.parts;
  a.dw.plane_a = size_t(s.T) * p.Ep;
  a.dw.b = x;
  a.dw.krows = s.T;
  a.dw.M = E;
  a.dw.Kdim = s.T;
  a.dw.chunk = p.chunk;
  a.dw.splits = p.splits;
  float* part = reinterpret_cast<float*>(w + p.part);
  a.dw.c = !dw ? nullptr : p.splits > 1 ? part : dw;
  if (p.form == kRbBig) launch_products<kRbBig, true>(a, st);
  else if (p.form == kRbSmall) bf ? launch_products<kRbSmall, true>(a, st) : launch_products<kRbSmall, false>(a, st);
  else bf ? launch_products<kRbFew, true>(a, st) : launch_products<kRbFew, false>(a, st);
  if (dw && p.splits > 1) {
    const size_t n = size_t(E) * s.d;
    hipLaunchKernelGGL(sum_parts_kernel, dim3(unsigned((n / 4 + 255) / 256)), dim3(256), 0, st, part, dw, p.splits, n);
  }
  return hipGetLastError();
}

}  // namespace lcm
