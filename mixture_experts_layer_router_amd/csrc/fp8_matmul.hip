// Product of two block-FP8 matrices, C = A B^T (include/lc_moe_block.h).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies E4M3 codes and applies one E8M0 scale per row
// of A and of B and 32 reduction elements, taken from the lane that holds them.  The products
// are exact; the instruction adds its 64 products and the accumulator with about 12 bits below
// the largest addend, which the result's rounding to bf16 (8 bits) covers.
//
// A stage is 128 reduction columns, one scale block: BM + BN rows of 128 bytes, loaded into LDS
// directly, 16-byte piece c of row r in slot c ^ (r & 7) (eight lanes of a fragment read then
// fall on all banks), and the scale bytes of the tile's rows, laid out so that one word holds
// those of a lane's rows in four row blocks.
#include "block.h"
#include "lds_dma.h"
#include "train.h"

namespace lcm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct MatmulArgs {
  const unsigned char *a, *b;  // codes
  const unsigned char *as, *bs;
  size_t lda, ldb, las, lbs;
  const bf16_t* add;
  bf16_t* out;
  float* part;
  int M, N, nkb, chunk, splits, mt, nt;
};

// WM x WN waves; a wave holds MB x NB blocks of 32 x 32.
template <int WM, int WN, int MB, int NB, int NST>
__global__ __launch_bounds__(WM* WN * 64) void matmul_fp8_kernel(MatmulArgs p) {
  constexpr int NW = WM * WN, BM = WM * MB * 32, BN = WN * NB * 32;
  constexpr int STAGE = (BM + BN) * 128 + 512;  // codes of A, of B, 256 scale bytes of each
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // loads a wave and stage: 8 rows each
  constexpr int PER = LA + LB + 1;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0 && NW % 2 == 0, "");
  __shared__ __attribute__((aligned(1024))) unsigned char smem[NST * STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // tiles in order along the rows first; every XCD takes a run of them
  const int tiles = p.mt * p.nt, per_xcd = (tiles * p.splits + 7) / 8;
  const int unit = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per_xcd || unit >= tiles * p.splits) return;
  const int split = unit / tiles, tile = unit % tiles;
  const int m0 = tile / p.nt * BM, n0 = tile % p.nt * BN;
  const int k0 = split * p.chunk, nk = min(p.chunk, p.nkb - k0);

  // sources: rows past the matrix read its last row and are not stored
  uint32_t off[LA + LB];
#pragma unroll
  for (int i = 0; i < LA + LB; ++i) {
    const bool isb = i >= LA;
    const int r = (isb ? (i - LA) * NW + wave : i * NW + wave) * 8 + (lane >> 3);
    const int last = (isb ? p.N - n0 : p.M - m0) - 1;
    off[i] = uint32_t(min(r, last)) * uint32_t(isb ? p.ldb : p.lda) + (((lane & 7) ^ (r & 7)) << 4);
  }
  const unsigned char* abase = p.a + size_t(m0) * p.lda + size_t(k0) * 128;
  const unsigned char* bbase = p.b + size_t(n0) * p.ldb + size_t(k0) * 128;
  const unsigned char* sbase = (wave & 1) ? p.bs + size_t(k0) * p.lbs + n0 : p.as + size_t(k0) * p.las + m0;
  const size_t sstep = (wave & 1) ? p.lbs : p.las;
  auto issue = [&](int kt, int slot) {
    unsigned char* st = smem + slot * STAGE;
#pragma unroll
    for (int i = 0; i < LA; ++i) dma16(abase + size_t(kt) * 128 + off[i], st + (i * NW + wave) * 1024);
#pragma unroll
    for (int i = 0; i < LB; ++i) dma16(bbase + size_t(kt) * 128 + off[LA + i], st + BM * 128 + (i * NW + wave) * 1024);
    // scales: every other wave A's, the rest B's (the same bytes: one count for all waves)
    __builtin_amdgcn_global_load_lds(sbase + size_t(kt) * sstep + lane * 4,
                                     (lds_void*)(st + (BM + BN) * 128 + (wave & 1) * 256), 4, 0, 0);
  };

  f32x16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int npro = nk < NST ? nk : NST;
  for (int s = 0; s < npro; ++s) issue(s, s);
  const int l32 = lane & 31, h = lane >> 5;
  // LDS reads are of bf16 vectors throughout: reads of other types wait for every load in flight
  auto frag = [&](const unsigned char* rows, int r, int ks) {
    const int c = ks * 4 + h * 2;
    const unsigned char* at = rows + r * 128;
    const i32x4 lo = __builtin_bit_cast(i32x4, *reinterpret_cast<const bf16x8*>(at + ((c ^ (r & 7)) << 4)));
    const i32x4 hi = __builtin_bit_cast(i32x4, *reinterpret_cast<const bf16x8*>(at + (((c + 1) ^ (r & 7)) << 4)));
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  // the scale bytes of the lane's row in row block b (of 32 rows) of the tile
  auto scale = [&](const unsigned char* sc, int b) {
    const uint32_t w = __builtin_bit_cast(uint32_t, *reinterpret_cast<const bf16x2*>(sc + (b >> 2) * 128 + l32 * 4));
    return int(w >> (8 * (b & 3)) & 0xFF);
  };
  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    const int newest = kt + NST - 1 < nk - 1 ? kt + NST - 1 : nk - 1;
    wait_vmcnt((newest - kt) * PER);
    block_barrier();
    const unsigned char* st = smem + slot * STAGE;
    const unsigned char* sc = st + (BM + BN) * 128;
    int sa[MB], sb[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) sa[i] = scale(sc, wm * MB + i);
#pragma unroll
    for (int j = 0; j < NB; ++j) sb[j] = scale(sc + 256, wn * NB + j);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      i32x8 fa[MB], fb[NB];
#pragma unroll
      for (int i = 0; i < MB; ++i) fa[i] = frag(st, (wm * MB + i) * 32 + l32, ks);
#pragma unroll
      for (int j = 0; j < NB; ++j) fb[j] = frag(st + BM * 128, (wn * NB + j) * 32 + l32, ks);
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 0, 0, 0, sa[i], 0, sb[j]);
    }
    wait_lds_reads();
    block_barrier();
    if (kt + NST < nk) issue(kt + NST, slot);
    slot = slot + 1 == NST ? 0 : slot + 1;
  }

  // column lane & 31, rows 8 (r / 4) + 4 (lane / 32) + r % 4 of a block
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int col = n0 + (wn * NB + j) * 32 + l32;
      if (col >= p.N) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = m0 + (wm * MB + i) * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (row >= p.M) continue;
        const size_t at = size_t(row) * p.N + col;
        if (p.part) {
          p.part[size_t(split) * p.M * p.N + at] = acc[i][j][r];
        } else {
          const float v = p.add ? acc[i][j][r] + bf2f(p.add[at]) : acc[i][j][r];
          p.out[at] = bf16_t(pack_bf16(v, 0.f));
        }
      }
    }
}

// out = sum of the pieces in order (+ add), 8 elements a thread.
__global__ __launch_bounds__(256) void matmul_join_kernel(const float* __restrict__ part, int splits, size_t n,
                                                          const bf16_t* add, bf16_t* out) {
  const size_t i = (size_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float4 a = *reinterpret_cast<const float4*>(part + s * n + i);
    const float4 b = *reinterpret_cast<const float4*>(part + s * n + i + 4);
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
  if (add) {
    const uint4 q = *reinterpret_cast<const uint4*>(add + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] += __uint_as_float(w[j] << 16);
      v[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  *reinterpret_cast<uint4*>(out + i) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

MatmulPlan plan_matmul_fp8(int M, int N, int K) {
  MatmulPlan p{};
  const int nkb = (K + 127) / 128;
  const size_t t256 = size_t((M + 255) / 256) * ((N + 255) / 256), t128 = size_t((M + 127) / 128) * ((N + 127) / 128);
  p.form = t256 >= 192 ? 0 : 1;
  const size_t tiles = p.form == 0 ? t256 : t128;
  size_t want = p.form == 0 ? 1 : 512 / tiles;
  if (want > size_t(nkb)) want = nkb;
  if (want < 1) want = 1;
  p.chunk = int((nkb + want - 1) / want);
  p.splits = (nkb + p.chunk - 1) / p.chunk;
  p.part = 0;
  p.total = p.splits > 1 ? align256(size_t(p.splits) * M * N * 4) : 256;
  return p;
}

hipError_t launch_matmul_fp8(int M, int N, int K, const MatmulPlan& p, void* ws, const void* a, const void* b,
                             const void* add, void* out, hipStream_t st) {
  const Fp8Mat am = plan_fp8_mat(M, K), bm = plan_fp8_mat(N, K);
  const unsigned char *ac = static_cast<const unsigned char*>(a), *bc = static_cast<const unsigned char*>(b);
  MatmulArgs g{ac, bc, ac + am.scales, bc + bm.scales, am.ldc, bm.ldc, am.lds, bm.lds,
               static_cast<const bf16_t*>(add), static_cast<bf16_t*>(out), p.splits > 1 ? static_cast<float*>(ws) : nullptr,
               M, N, am.nkb, p.chunk, p.splits, 0, 0};
  const int bt = p.form == 0 ? 256 : 128;
  g.mt = (M + bt - 1) / bt;
  g.nt = (N + bt - 1) / bt;
  const unsigned grid = unsigned((size_t(g.mt) * g.nt * p.splits + 7) / 8 * 8);
  if (p.form == 0) matmul_fp8_kernel<2, 4, 4, 2, 2><<<dim3(grid), dim3(512), 0, st>>>(g);
  else matmul_fp8_kernel<2, 2, 2, 2, 2><<<dim3(grid), dim3(256), 0, st>>>(g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const size_t n = size_t(M) * N;
  matmul_join_kernel<<<dim3(unsigned((n / 8 + 255) / 256)), dim3(256), 0, st>>>(g.part, p.splits, n, g.add, g.out);
  return hipGetLastError();
}

}  // namespace lcm
