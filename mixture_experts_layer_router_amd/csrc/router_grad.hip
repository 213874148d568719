// Backward of the router: the softmax's gradient from the gates' gradients, then the two
// products with the router weight and with the tokens (formulas in
// include/lc_moe_train.h).
//
//   dlogits_kernel   one wave per token: dlogits in fp32, cut into three bf16 parts
//   parts_kernel     W_r (and fp32 tokens) cut into parts
//   product_kernel   dx = dlogits W_r (+ dx_add) and dW = dlogits^T x on the matrix cores
//   sum_parts_kernel the pieces of dW's reduction over the tokens, added in order
#include <type_traits>

#include "train.h"
#include "lanes.h"
#include "lds_dma.h"
#include "logit_row.h"

namespace lcm {

// v = h + m + l exactly but for the last of its 24 significant bits (each part keeps 8, the
// remainders are exact in fp32).
__device__ __forceinline__ void cut3(float v, bf16_t (&o)[3]) {
  o[0] = f2bf(v);
  const float r1 = v - bf2f(o[0]);
  o[1] = f2bf(r1);
  o[2] = f2bf(r1 - bf2f(o[1]));
}

// ---------------------------------------------------------------------------------------
// dlogits of one token per wave, the row in its registers as in logit_row.h.  The picks'
// gradients are added in pick order by the lane that holds the expert.
// ---------------------------------------------------------------------------------------
template <int EPL, int V>
__global__ __launch_bounds__(256) void dlogits_kernel(const float* __restrict__ logits,
                                                      const int32_t* __restrict__ idx,
                                                      const float* __restrict__ dgate, const float* aux, int T, int E,
                                                      int K, int Ep, float* out, bf16_t* __restrict__ parts) {
  constexpr int J = EPL / V;  // runs of 64 V experts
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  float v[EPL], ax[EPL];
  if (dgate) load_row<EPL, V>(logits + size_t(t) * E, E, lane, -INFINITY, v);
  if (aux) load_row<EPL, V>(aux + size_t(t) * E, E, lane, 0.f, ax);
  if (dgate) {
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
        pe = idx[size_t(t) * K + k0 + lane];
        pg = dgate[size_t(t) * K + k0 + lane];
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
  if (aux) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] += ax[i];
  }
  const size_t plane = size_t(T) * Ep;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = (j * 64 + lane) * V;
    if (e >= Ep) continue;
    bf16_t* dst = parts + size_t(t) * Ep + e;
    if constexpr (V == 4) {
      bf16_t h[4][3];
#pragma unroll
      for (int w = 0; w < 4; ++w) cut3(e < E ? v[4 * j + w] : 0.f, h[w]);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<uint2*>(dst + q * plane) =
            make_uint2(h[0][q] | (uint32_t(h[1][q]) << 16), h[2][q] | (uint32_t(h[3][q]) << 16));
      if (out && e < E)
        *reinterpret_cast<float4*>(out + size_t(t) * E + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      bf16_t h[3];
      cut3(e < E ? v[j] : 0.f, h);
#pragma unroll
      for (int q = 0; q < 3; ++q) dst[q * plane] = h[q];
      if (out && e < E) out[size_t(t) * E + e] = v[j];
    }
  }
}

// Parts of a matrix [R][C] fp32 (C a multiple of 4): NP planes [Rp][Cp], zeros past R and C.
// Thread: 4 columns.  Also the 16 zero bytes that operand chunks past the data are read from.
template <int NP>
__global__ __launch_bounds__(256) void parts_kernel(const float* __restrict__ src, bf16_t* __restrict__ dst, int R,
                                                    int C, size_t n4, int Cp, uint4* __restrict__ zero) {
  const size_t i = size_t(blockIdx.x) * 256 + threadIdx.x;
  if (i == 0) *zero = make_uint4(0, 0, 0, 0);
  if (i >= n4) return;
  const size_t r = i / (Cp / 4);
  const int c = int(i - r * (Cp / 4)) * 4;
  const float4 v = r < size_t(R) && c < C ? *reinterpret_cast<const float4*>(src + r * C + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  bf16_t h[4][3];
  cut3(v.x, h[0]);
  cut3(v.y, h[1]);
  cut3(v.z, h[2]);
  cut3(v.w, h[3]);
#pragma unroll
  for (int q = 0; q < NP; ++q)
    *reinterpret_cast<uint2*>(dst + q * n4 * 4 + i * 4) =
        make_uint2(h[0][q] | (uint32_t(h[1][q]) << 16), h[2][q] | (uint32_t(h[3][q]) << 16));
}

// ---------------------------------------------------------------------------------------
// C[M][N] = sum over pairs of parts (a, b) of A_a B_b, fp32 accumulation on
// v_mfma_f32_32x32x16_bf16.  One stage holds 32 reduction steps of NA parts of A and NB
// parts of B, so a loaded part serves every product it takes part in: with pairs
// a + b < max(NA, NB) (h h, h m, m h of two parts each; h x, m x, l x of three and one; the
// six largest of three and three) a stage's (NA + NB) operand tiles carry 3 or 6 products.
//   DX: A(m, k) = dlogits parts, row m, K-contiguous; B(k, n) = W_r parts, row k.
//   DW: A(m, k) = dlogits parts, row k (tokens), M-contiguous; B(k, n) = tokens, row k.
// Tile BM x BN, 64 x (BN / 2) outputs per wave, BM / 32 waves, a two-stage ring in LDS
// filled by direct global->LDS loads.  Operands whose output index is contiguous lie in LDS
// as in memory ([32 steps][columns]) and are read by the transposing LDS read; 16-byte chunk
// c of row r sits in the 32-byte granule (c / 2) ^ 2 (r % 4), which spreads the four rows of
// a read over the banks.  K-contiguous rows are 64 bytes, chunk c in slot c ^ swz4(r).
// ---------------------------------------------------------------------------------------
struct ProdArgs {
  const bf16_t* a;  // [NA][T][Ep]
  const bf16_t* b;  // DX: [NB][Ep][ldb]; DW: [NB][T][ldb]
  size_t plane_a, plane_b;
  const bf16_t* zero;
  const void* add;
  void* c;
  int M, N, Kdim, lda, ldb;
  int chunk;        // reduction steps of a piece (a multiple of 32)
  int n_mt, n_nt, splits;
};

template <bool DX, int BM, int BN, int NA, int NB, typename Tc>
__global__ __launch_bounds__(BM * 2, 1) void product_kernel(ProdArgs p) {
  constexpr int BK = 32, WAVES = BM / 32, WN = 2, WC = BN / WN;  // wave tile: 64 x WC
  constexpr int NBL = WC / 32;                                  // 32-wide column blocks of a wave
  constexpr int A_OP = BM * BK * 2, B_OP = BN * BK * 2;          // bytes of one part in a stage
  constexpr int STAGE = NA * A_OP + NB * B_OP;
  constexpr int NP = NA > NB ? NA : NB;
  constexpr int LA = A_OP / 1024 / WAVES, LB = B_OP / 1024 / WAVES;  // direct loads of a wave per part
  static_assert(A_OP % (1024 * WAVES) == 0 && B_OP % (1024 * WAVES) == 0, "whole loads");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * STAGE];

  // unit: groups of 4 M-tiles, in a group column tiles, in them its M-tiles; each XCD takes a
  // contiguous eighth, so workgroups side by side share operand rows in its L2
  const int U = p.n_mt * p.n_nt * p.splits, per = (U + 7) >> 3, slot_w = blockIdx.x >> 3;
  if (slot_w >= per) return;
  const int u = (blockIdx.x & 7) * per + slot_w;
  if (u >= U) return;
  const int tiles = p.n_mt * p.n_nt, sp = u / tiles;
  int r0 = u - sp * tiles;
  const int grp = r0 / (4 * p.n_nt);
  r0 -= grp * 4 * p.n_nt;
  const int gm = p.n_mt - grp * 4 < 4 ? p.n_mt - grp * 4 : 4;
  const int m0 = (grp * 4 + r0 % gm) * BM, n0 = (r0 / gm) * BN;
  const int kbeg = sp * p.chunk, kend = kbeg + p.chunk < p.Kdim ? kbeg + p.chunk : p.Kdim;
  const int nk = (kend - kbeg + BK - 1) / BK;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // a wave's load i of an operand with contiguous columns (BC of them) fills bytes
  // 1024 (wave + WAVES i) of its part: RPL rows of 2 BC bytes
  auto col_load = [&](const bf16_t* src, size_t plane, int np, int op_bytes, int BC, int n_loads, int k0, int c0, int ld,
                      int cols, unsigned char* dst) {
    const int rpl = 512 / BC, cpr = BC / 8;  // rows of a load, 16-byte chunks of a row
    for (int i = 0; i < n_loads; ++i) {
      const int kr = rpl * (wave + WAVES * i) + lane / cpr, sl = lane % cpr;
      const int ch = 2 * ((sl >> 1) ^ (2 * (kr & 3))) + (sl & 1);
      const int k = k0 + kr, c = c0 + ch * 8;
      const bool in = k < kend && c < cols;
      const bf16_t* g = src + size_t(k) * ld + c;
      for (int q = 0; q < np; ++q)
        dma16(in ? g + q * plane : p.zero, dst + q * op_bytes + (wave + WAVES * i) * 1024);
    }
  };
  auto issue = [&](int kt) {
    unsigned char* st = smem + (kt & 1) * STAGE;
    const int k0 = kbeg + kt * BK;
    if constexpr (DX) {
#pragma unroll
      for (int i = 0; i < LA; ++i) {
        const int r = 16 * (wave + WAVES * i) + (lane >> 2);
        const int m = m0 + r < p.M ? m0 + r : m0;  // rows past M repeat a valid row; never stored
        const bf16_t* g = p.a + size_t(m) * p.lda + k0 + ((lane & 3) ^ swz4(r)) * 8;
#pragma unroll
        for (int q = 0; q < NA; ++q) dma16(g + q * p.plane_a, st + q * A_OP + (wave + WAVES * i) * 1024);
      }
    } else {
      col_load(p.a, p.plane_a, NA, A_OP, BM, LA, k0, m0, p.lda, p.lda, st);
    }
    col_load(p.b, p.plane_b, NB, B_OP, BN, LB, k0, n0, p.ldb, p.ldb, st + NA * A_OP);
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

  if (nk > 0) issue(0);
  for (int kt = 0; kt < nk; ++kt) {
    LCM_WAIT_VMCNT(0);  // stage kt landed (stage kt + 1 is not issued yet)
    wait_lds_reads();
    block_barrier();    // every wave's loads of stage kt visible; stage kt - 1 read by all
    if (kt + 1 < nk) issue(kt + 1);
    const unsigned char* st = smem + (kt & 1) * STAGE;
    const unsigned char* sb = st + NA * A_OP;
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      bf16x8 fa[NA][2], fb[NB][NBL];
      if constexpr (DX) {
#pragma unroll
        for (int q = 0; q < NA; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            fa[q][i] = *reinterpret_cast<const bf16x8*>(st + q * A_OP + (wm * 64 + i * 32 + l32) * 64 +
                                                        (((ks / 8 + khalf) ^ swz4(l32)) << 4));
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
#pragma unroll
      for (int q = 0; q < NB; ++q) {
        if constexpr (NBL == 4) {
          uint32_t ad[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) ad[j] = tr_addr(sb + q * B_OP, BN * 2, wn * WC + 32 * j, ks);
          tr8(std::integral_constant<int, BN * 2>{}, ad, fb[q]);
        } else {
          static_assert(NBL == 2, "wave tiles of 64 or 128 columns");
          tr4(std::integral_constant<int, BN * 2>{}, tr_addr(sb + q * B_OP, BN * 2, wn * WC, ks),
              tr_addr(sb + q * B_OP, BN * 2, wn * WC + 32, ks), fb[q][0], fb[q][1]);
        }
      }
#pragma unroll
      for (int qa = 0; qa < NA; ++qa)
#pragma unroll
        for (int qb = 0; qb < NB; ++qb) {
          if (qa + qb >= NP) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NBL; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[qa][i], fb[qb][j], acc[i][j], 0, 0, 0);
        }
    }
  }

  // 32x32 D layout: column lane % 32, rows 8 (r / 4) + 4 (lane / 32) + r % 4; a transpose among
  // four lanes gives each lane one row of 4 columns
  const int q4 = lane & 3;
  Tc* out = static_cast<Tc*>(p.c) + (DX ? 0 : size_t(sp) * p.M * p.N);
  const Tc* add = static_cast<const Tc*>(p.add);
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
        const int m = m0 + wm * 64 + i * 32 + 8 * rq + 4 * khalf + q4;
        const int n = n0 + wn * WC + j * 32 + (lane & 28);
        if (m >= p.M || n >= p.N) continue;
        const size_t o = size_t(m) * p.N + n;
        if constexpr (sizeof(Tc) == 2) {
          if (add) {
            const uint2 q = *reinterpret_cast<const uint2*>(add + o);
            w[0] += __uint_as_float(q.x << 16);
            w[1] += __uint_as_float(q.x & 0xFFFF0000u);
            w[2] += __uint_as_float(q.y << 16);
            w[3] += __uint_as_float(q.y & 0xFFFF0000u);
          }
          *reinterpret_cast<uint2*>(out + o) =
              make_uint2(f2bf(w[0]) | (uint32_t(f2bf(w[1])) << 16), f2bf(w[2]) | (uint32_t(f2bf(w[3])) << 16));
        } else {
          if (add) {
            const float4 q = *reinterpret_cast<const float4*>(add + o);
            w[0] += q.x, w[1] += q.y, w[2] += q.z, w[3] += q.w;
          }
          *reinterpret_cast<float4*>(out + o) = make_float4(w[0], w[1], w[2], w[3]);
        }
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

template <bool DX, int BM, int BN, int NA, int NB, typename Tc>
static void product(ProdArgs p, hipStream_t st) {
  p.n_mt = (p.M + BM - 1) / BM;
  p.n_nt = (p.N + BN - 1) / BN;
  const size_t units = size_t(p.n_mt) * p.n_nt * p.splits;
  hipLaunchKernelGGL((product_kernel<DX, BM, BN, NA, NB, Tc>), dim3(unsigned((units + 7) / 8 * 8)), dim3(BM * 2), 0, st, p);
}

template <bool BF>
static void products(const lc_moe_shape& s, const RouterBwPlan& pl, char* w, const void* x, const float* w_router,
                     const void* add, void* dx, float* dw, hipStream_t st) {
  typedef typename std::conditional<BF, bf16_t, float>::type Tx;
  constexpr int BN = BF ? kRbBig : kRbSmall, W = BF ? 2 : 3, X = BF ? 1 : 3;
  const int E = s.N + s.Z;
  bf16_t* wp = reinterpret_cast<bf16_t*>(w + pl.wp);
  bf16_t* xp = reinterpret_cast<bf16_t*>(w + pl.xp);
  uint4* zero = reinterpret_cast<uint4*>(w + pl.zero);
  const size_t nw = dx ? size_t(pl.Ep) * pl.dp / 4 : 0, nx = size_t(s.T) * pl.dp / 4;
  hipLaunchKernelGGL((parts_kernel<W>), dim3(unsigned(nw / 256 + 1)), dim3(256), 0, st, w_router, wp, E, s.d, nw, pl.dp, zero);
  ProdArgs p{};
  p.a = reinterpret_cast<const bf16_t*>(w + pl.dl);
  p.plane_a = size_t(s.T) * pl.Ep;
  p.lda = pl.Ep;
  p.ldb = pl.dp;
  p.zero = reinterpret_cast<const bf16_t*>(zero);
  p.N = s.d;
  if (dx) {
    p.b = wp;
    p.plane_b = size_t(pl.Ep) * pl.dp;
    p.M = s.T;
    p.Kdim = p.chunk = pl.Ep;
    p.splits = 1;
    p.add = add;
    p.c = dx;
    if (pl.dx_big) product<true, kRbBig, BN, W, W, Tx>(p, st);
    else product<true, kRbSmall, kRbSmall, W, W, Tx>(p, st);
  }
  if (dw) {
    if (!BF)
      hipLaunchKernelGGL((parts_kernel<3>), dim3(unsigned((nx + 255) / 256)), dim3(256), 0, st,
                         static_cast<const float*>(x), xp, s.T, s.d, nx, pl.dp, zero);
    p.b = BF ? static_cast<const bf16_t*>(x) : xp;
    p.plane_b = size_t(s.T) * pl.dp;
    p.M = E;
    p.Kdim = s.T;
    p.chunk = pl.chunk;
    p.splits = pl.splits;
    p.add = nullptr;
    p.c = pl.splits > 1 ? reinterpret_cast<float*>(w + pl.part) : dw;
    if (pl.dw_big) product<false, kRbBig, BN, 3, X, float>(p, st);
    else product<false, kRbSmall, kRbSmall, 3, X, float>(p, st);
    if (pl.splits > 1) {
      const size_t n = size_t(E) * s.d;
      hipLaunchKernelGGL(sum_parts_kernel, dim3(unsigned((n / 4 + 255) / 256)), dim3(256), 0, st,
                         reinterpret_cast<const float*>(w + pl.part), dw, pl.splits, n);
    }
  }
}

hipError_t launch_router_backward(const lc_moe_shape& s, const RouterBwPlan& p, void* ws, const void* x,
                                  const float* w_router, const float* logits, const int32_t* idx,
                                  const float* dgate, const float* aux, const void* dx_add, void* dx, float* dw,
                                  float* dlogits, hipStream_t st) {
  const int E = s.N + s.Z, epl = (E + 63) / 64;
  char* w = static_cast<char*>(ws);
  bf16_t* parts = reinterpret_cast<bf16_t*>(w + p.dl);
#define LCM_DL(n, v)                                                                                                  \
  hipLaunchKernelGGL((dlogits_kernel<n, v>), dim3((s.T + 3) / 4), dim3(256), 0, st, logits, idx, dgate, aux, s.T, E, \
                     s.K, p.Ep, dlogits, parts)
  if (E % 4 == 0) {
    if (epl <= 4) LCM_DL(4, 4);
    else if (epl <= 8) LCM_DL(8, 4);
    else if (epl <= 12) LCM_DL(12, 4);
    else if (epl <= 16) LCM_DL(16, 4);
    else if (epl <= 32) LCM_DL(32, 4);
    else LCM_DL(64, 4);
  } else {
    if (epl <= 2) LCM_DL(2, 1);
    else if (epl <= 4) LCM_DL(4, 1);
    else if (epl <= 8) LCM_DL(8, 1);
    else if (epl <= 16) LCM_DL(16, 1);
    else if (epl <= 32) LCM_DL(32, 1);
    else LCM_DL(64, 1);
  }
#undef LCM_DL
  if (s.dtype == LC_MOE_BF16) products<true>(s, p, w, x, w_router, dx_add, dx, dw, st);
  else products<false>(s, p, w, x, w_router, dx_add, dx, dw, st);
  return hipGetLastError();
}

}  // namespace lcm
