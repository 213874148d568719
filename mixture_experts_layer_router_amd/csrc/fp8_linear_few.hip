// y = Q(x) W^T for few tokens or small matrices, x quantised on the way (include/lc_moe_block.h).
//
// With few tokens the weight's bytes bound the product, and next to them every launch counts.  A wavefront
// multiplies all tokens with 32 rows of W over whole runs of 128 columns by itself: it loads the codes
// straight into the operands' registers and the tokens' bf16 values beside them, finds each row's largest
// among the 128 (a lane holds 32 of them, three others the rest) and converts them in place.  So nothing
// passes through LDS, and no wave waits for another, until the eight waves of a workgroup add their sums up
// in order.  Within a run the order of the columns does not matter as long as both operands have the same:
// lane (r, g) of 16 x 4 holds the 16-byte pieces g and 4 + g of row r's codes, so that four lanes read 64
// neighbouring bytes, and the 16 x 16 x 128 product takes a run at once (32 x 32 x 64 touched twice as many
// cache lines a load: 15.9 -> 14.1 us at T = 16, k = n = 6144).
//
// Kernel times by trace, against those of the launch that quantises x and the one or two that multiply
// (fp8_matmul.hip), us; (a call takes 9.5 us of the host's time unless a graph holds it):
//   k = n = 6144   T = 1: 9.8 (3.9 TB/s of W; 15.5)   16: 13.6 (18.7)   32: 20.4 (20.1)
//   k = n = 1024   T = 1: 3.9 (9.5)                   64:  4.8 (10.2)  400:  8.5 (10.6)   777: 14.6 (10.8)
//   k = n =  520   T = 1: 3.7 (8.3)                   64:  4.0 (9.0)   400:  4.6 (10.0)   777:  6.2 (10.1)
// (T = 32 and 777 of the wider ones go the other way, by the figures below.)
// What bounds it is a CU's loads: a run of 32 rows of W and of 16 tokens is 8 KB, of 64 tokens 20 KB, and
// every workgroup reads x anew.  linear_few weighs the two ways by kFewForms and the product's own figures.
#include "block.h"
#include "train.h"

namespace lcm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct FewArgs {
  const bf16_t* x;
  const unsigned char *w, *ws;  // codes, scales
  size_t ldw, lws;
  const bf16_t* add;
  bf16_t* y;
  float* part;  // [splits][T][n], or null: no pieces
  int T, k, n, nkb, chunk, tiles;
};

// The largest of the absolute values in v (bf16 pairs) and m.
__device__ __forceinline__ u16x2 abs_max(u16x2 m, uint32_t v) {
  return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu));
}
// Smallest e with a bf16 value of these bits <= 448 * 2^e = 1.75 * 2^(e + 8), not below -127; 0 for 0.
__device__ __forceinline__ int fp8_exp_of_bf16(int bits) {
  const int e = (bits >> 7) - 135 + ((bits & 0x7F) > 0x60 ? 1 : 0);
  return bits == 0 ? 0 : max(e, -127);
}

constexpr int kFewWaves = 8;  // wavefronts of a workgroup, among which its runs go in turn
// Blocks of tokens, and what they take (us, measured): a run of 128 columns on a CU, and one more workgroup
// on it.  (64, 1024, 1024): 4.7 us in blocks of 16 tokens, 5.7 of 32, 7.9 of 64; (777, 520, 520): 7.5, 6.8, 5.9.
struct FewForm {
  int tokens;
  float run, next;
};
constexpr FewForm kFewForms[] = {{16, 0.2f, 0.5f}, {32, 0.33f, 0.8f}, {64, 0.6f, 1.3f}};

// MB: blocks of 16 tokens.
template <int MB>
__global__ __launch_bounds__(kFewWaves * 64) void linear_few_kernel(FewArgs p) {
  constexpr int ROWS = MB * 16, NB = 2, COLS = NB * 16, PIECES = COLS / 4, WAVES = kFewWaves;
  // the waves' sums on their way together: 16-byte piece c of row r is in slot c ^ (r % PIECES)
  __shared__ __attribute__((aligned(16))) float sums[WAVES][ROWS][COLS];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x % p.tiles, split = blockIdx.x / p.tiles, t0 = blockIdx.y * ROWS;
  const int n0 = tile * COLS, k0 = split * p.chunk, k1 = min(k0 + p.chunk, p.nkb);

  const unsigned char* wrow[NB];  // rows past the matrix read its last row and are not stored
#pragma unroll
  for (int j = 0; j < NB; ++j) wrow[j] = p.w + size_t(min(n0 + j * 16 + l16, p.n - 1)) * p.ldw + g * 16;
  const bf16_t* xrow[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) xrow[i] = p.x + size_t(min(t0 + i * 16 + l16, p.T - 1)) * p.k + g * 16;

  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 nw[NB][2], nx[MB][4];
  uint32_t ns[2] = {0, 0};
  auto load = [&](int kb) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) nw[j][q] = *reinterpret_cast<const u32x4*>(wrow[j] + size_t(kb) * 128 + q * 64);
    // the exponents of the rows n0 & ~127 on: those of blocks of 32 in the bytes of a word
#pragma unroll
    for (int s = 0; s < 2; ++s)
      ns[s] = *reinterpret_cast<const uint32_t*>(p.ws + size_t(kb) * p.lws + (n0 & ~127) + (s * 16 + l16) * 4);
    const int col = kb * 128 + g * 16;
    if (kb * 128 + 128 <= p.k) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          nx[i][q] = *reinterpret_cast<const u32x4*>(xrow[i] + size_t(kb) * 128 + q / 2 * 64 + q % 2 * 8);
    } else {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          nx[i][q] = u32x4{0, 0, 0, 0};
          if (col + q / 2 * 64 + q % 2 * 8 < p.k)
            nx[i][q] = *reinterpret_cast<const u32x4*>(xrow[i] + size_t(kb) * 128 + q / 2 * 64 + q % 2 * 8);
        }
    }
  };
  int kb = k0 + wave;
  if (kb < k1) load(kb);
  for (; kb < k1; kb += WAVES) {
    i32x8 fa[MB], fb[NB];
    int sa[MB];
    const int sb[2] = {int(ns[0] >> ((n0 & 127) / 4)), int(ns[1] >> ((n0 & 127) / 4))};
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) fb[j][e] = int(nw[j][e / 4][e % 4]);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      u16x2 m = {0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = abs_max(m, nx[i][q][e]);
      const int bits = int(max_of_rows(max(uint32_t(m[0]), uint32_t(m[1]))));
      sa[i] = fp8_exp_of_bf16(bits) + 127;
      const float unit = __uint_as_float(uint32_t(sa[i]) << 23);  // the conversion reads the exponent alone
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // a register of four codes: two pairs of values
        const uint32_t lo = nx[i][e / 2][e % 2 * 2], hi = nx[i][e / 2][e % 2 * 2 + 1];
        i16x2 c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, lo), unit, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, hi), unit, true);
        fa[i][e] = __builtin_bit_cast(int, c);
      }
    }
    if (kb + WAVES < k1) load(kb + WAVES);  // beside the products
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      acc[i][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[0], fa[i], acc[i][0], 0, 0, 0, sb[0], 0, sa[i]);
      acc[i][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[1], fa[i], acc[i][1], 0, 0, 0, sb[1], 0, sa[i]);
    }
  }
  // lane: token l16, columns 4 g on of a block
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<float4*>(&sums[wave][i * 16 + l16][((j * 4 + g) ^ (l16 % PIECES)) * 4]) =
          make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  __syncthreads();
  for (int i = tid; i < ROWS * PIECES; i += WAVES * 64) {
    const int r = i / PIECES, c = i % PIECES, col = n0 + c * 4;
    if (t0 + r >= p.T || col >= p.n) continue;
    const int slot = (c ^ (r % PIECES)) * 4;
    float4 f = *reinterpret_cast<const float4*>(&sums[0][r][slot]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(&sums[w][r][slot]);
      f.x += v.x, f.y += v.y, f.z += v.z, f.w += v.w;
    }
    const size_t at = size_t(t0 + r) * p.n + col;
    if (p.part) {
      *reinterpret_cast<float4*>(p.part + size_t(split) * p.T * p.n + at) = f;
      continue;
    }
    if (p.add) {
      const uint2 q = *reinterpret_cast<const uint2*>(p.add + at);
      f.x += __uint_as_float(q.x << 16), f.y += __uint_as_float(q.x & 0xFFFF0000u);
      f.z += __uint_as_float(q.y << 16), f.w += __uint_as_float(q.y & 0xFFFF0000u);
    }
    *reinterpret_cast<uint2*>(p.y + at) = make_uint2(pack_bf16(f.x, f.y), pack_bf16(f.z, f.w));
  }
}

// The blocks of tokens and the number of pieces of the columns that take the least by these figures.  Every
// wave of a piece has a run; pieces are joined by a second kernel.
LinearFewPlan plan_linear_few(int T, int k, int n) {
  LinearFewPlan p{};
  const int nkb = (k + 127) / 128, tiles = (n + 31) / 32;
  p.us = 1e30f;
  for (int f = 0; f < 3; ++f) {
    const FewForm& o = kFewForms[f];
    const int blocks = (T + o.tokens - 1) / o.tokens;
    if (blocks > 65535 || (f > 0 && T <= kFewForms[f - 1].tokens)) continue;
    for (int want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (want > 1 && want * kFewWaves > nkb) break;
      const int chunk = (nkb + want - 1) / want, splits = (nkb + chunk - 1) / chunk;
      if (splits != want) continue;
      const int64_t each = (int64_t(tiles) * blocks * splits + 255) / 256;  // workgroups of a CU
      float t = 3.2f + float(each) * float(chunk) * o.run + float(each - 1) * o.next;
      if (splits > 1) t += 2.f + float(splits) * float(T) * float(n) * 8 / 5e6f;
      if (t < p.us) p.us = t, p.form = f, p.chunk = chunk, p.splits = splits;
    }
  }
  p.total = p.splits > 1 ? align256(size_t(p.splits) * T * n * 4) : 256;
  return p;
}

// Against a launch that quantises the tokens (2.5 us and their bytes) and the product's.
bool linear_few(const LinearFewPlan& p, int T, int k, int n) {
  return p.us < 2.5f + float(T) * float(k) * 3 / 5e6f + plan_matmul_fp8(T, n, k).us;
}

hipError_t launch_linear_few(int T, int k, int n, const LinearFewPlan& p, void* ws, const void* x, const void* w,
                             const void* add, void* y, hipStream_t st) {
  const Fp8Mat m = plan_fp8_mat(n, k);
  const unsigned char* wc = static_cast<const unsigned char*>(w);
  const int tiles = (n + 31) / 32;
  const FewArgs a{static_cast<const bf16_t*>(x), wc, wc + m.scales, m.ldc, m.lds, static_cast<const bf16_t*>(add),
                  static_cast<bf16_t*>(y), p.splits > 1 ? static_cast<float*>(ws) : nullptr, T, k, n, m.nkb, p.chunk, tiles};
  const int tokens = kFewForms[p.form].tokens;
  const dim3 grid(unsigned(tiles * p.splits), unsigned((T + tokens - 1) / tokens)), block(kFewWaves * 64);
  if (p.form == 0) linear_few_kernel<1><<<grid, block, 0, st>>>(a);
  else if (p.form == 1) linear_few_kernel<2><<<grid, block, 0, st>>>(a);
  else linear_few_kernel<4><<<grid, block, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_matmul_join(a.part, p.splits, size_t(T) * n, a.add, a.y, st);
}

}  // namespace lcm
