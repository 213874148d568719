// bf16 matrices to block FP8 along their rows, their columns or both in one pass
// (include/lc_moe_block.h gives the layout).
//
// A workgroup takes a tile of 128 x 128; thread (rg, cg) = (tid / 16, tid % 16) holds rows
// 8 rg .. 8 rg + 7 and columns 8 cg .. 8 cg + 7 of it.  The codes of the transpose go through
// LDS, so that they too leave in whole 128-byte rows.  Memory bounds it: 16384 x 6144 bf16 along the rows
// takes 49-51 us (6 TB/s), both forms 81 (5 TB/s); dy both ways and x by its columns for a linear layer's
// gradient (n = 2048, k = 6144: 436 MB) 77 us (5.7 TB/s; 93 with the rows' maxima through LDS and those of
// the columns from 16 rows of it, 99 with the transpose's codes on few banks too).
#include "block.h"

namespace lcm {

// Smallest k with amax <= 448 * 2^k = 1.75 * 2^(k + 8), not below -127; 0 for amax = 0.
__device__ __forceinline__ int fp8_exp(float amax) {
  if (amax == 0.f) return 0;
  const int e = __builtin_amdgcn_frexp_expf(amax);  // amax = m 2^e, 0.5 <= m < 1
  const int k = __builtin_amdgcn_frexp_mantf(amax) <= 0.875f ? e - 9 : e - 8;
  return k > -127 ? k : -127;
}
// Four values over 2^k to E4M3 (nearest, ties to the even code), the first in the low byte.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d, int k) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(a, -k), ldexpf(b, -k), 0, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(c, -k), ldexpf(d, -k), q, true);
  return uint32_t(q);
}

struct QuantizeArgs {
  const bf16_t* x;
  int rows, cols;
  Fp8Mat m, mt;
  unsigned char *out, *out_t;
  int tiles;
};

// Tile number `tile` of one matrix.  BLOCK: one scale for the whole tile.  ROWS, COLS: the matrix, its
// transpose is written.
template <bool BLOCK, bool ROWS, bool COLS>
__device__ __forceinline__ void quantize_tile(const QuantizeArgs& q, int tile_index) {
  const bf16_t* __restrict__ x = q.x;
  const int rows = q.rows, cols = q.cols;
  const Fp8Mat m = q.m, mt = q.mt;
  unsigned char *__restrict__ out = q.out, *__restrict__ out_t = q.out_t;
  __shared__ float colmax[4][128];
  __shared__ float wmax[4];
  // Codes of the transpose: row stride 144, 16-byte piece p of row c in slot p ^ (c / 16): the 16 x 4 threads
  // of a wave, 8 rows and half a piece apart, then write to all banks alike (without: 8 of them to one).
  __shared__ __attribute__((aligned(16))) unsigned char tile[COLS ? 128 * 144 : 16];
  const int cb = tile_index % m.nkb, rb = tile_index / m.nkb;
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  const int r0 = rb * 128 + rg * 8, c0 = cb * 128 + cg * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (r0 + i < rows && c0 < cols) q = *reinterpret_cast<const uint4*>(x + size_t(r0 + i) * cols + c0);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i][2 * j] = __uint_as_float(w[j] << 16);
      v[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  int kr[8], kc[8];  // exponents of the thread's rows and columns
  if constexpr (BLOCK) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
    amax = __uint_as_float(max_of_rows(__float_as_uint(max_of_row(amax))));
    if ((tid & 63) == 0) wmax[tid >> 6] = amax;
    __syncthreads();
    const int k = fp8_exp(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) kr[i] = kc[i] = k;
  } else {
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
        kr[i] = fp8_exp(max_of_row(amax));
      }
    }
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i][j]));
        const uint32_t bits = max_of_rows(__float_as_uint(amax));  // (as numbers: not negative)
        if ((tid & 48) == 0) colmax[tid >> 6][cg * 8 + j] = __uint_as_float(bits);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float amax = 0.f;
#pragma unroll
        for (int g = 0; g < 4; ++g) amax = fmaxf(amax, colmax[g][cg * 8 + j]);
        kc[j] = fp8_exp(amax);
      }
    }
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i >= rows) continue;
      const uint32_t lo = fp8_codes(v[i][0], v[i][1], v[i][2], v[i][3], kr[i]);
      const uint32_t hi = fp8_codes(v[i][4], v[i][5], v[i][6], v[i][7], kr[i]);
      *reinterpret_cast<uint2*>(out + size_t(r0 + i) * m.ldc + c0) = make_uint2(lo, hi);
    }
    unsigned char* sc = out + m.scales + size_t(cb) * m.lds;
    if (cg == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sc[fp8_scale_at(r0 + i)] = static_cast<unsigned char>(r0 + i < rows ? kr[i] + 127 : 127);
    }
    // the bytes behind the last row's run of 128, and behind the last run
    if (rb == (rows + 127) / 128 - 1) {
      for (size_t i = size_t(rb + 1) * 128 + tid; i < m.lds; i += 256) sc[i] = 127;
      if (cb == m.nkb - 1) sc[m.lds + tid] = 127;
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t lo = fp8_codes(v[0][j], v[1][j], v[2][j], v[3][j], kc[j]);
      const uint32_t hi = fp8_codes(v[4][j], v[5][j], v[6][j], v[7][j], kc[j]);
      *reinterpret_cast<uint2*>(tile + (cg * 8 + j) * 144 + ((rg >> 1 ^ cg >> 1) << 4) + (rg & 1) * 8) = make_uint2(lo, hi);
    }
    unsigned char* sc = out_t + mt.scales + size_t(rb) * mt.lds;
    if (rg == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sc[fp8_scale_at(c0 + j)] = static_cast<unsigned char>(c0 + j < cols ? kc[j] + 127 : 127);
    }
    if (cb == m.nkb - 1) {
      for (size_t i = size_t(cb + 1) * 128 + tid; i < mt.lds; i += 256) sc[i] = 127;
      if (rb == mt.nkb - 1) sc[mt.lds + tid] = 127;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = tid + 256 * it, c = i >> 3, piece = i & 7;
      if (cb * 128 + c < cols)
        *reinterpret_cast<uint4*>(out_t + size_t(cb * 128 + c) * mt.ldc + rb * 128 + piece * 16) =
            *reinterpret_cast<const uint4*>(tile + c * 144 + (piece ^ c >> 4) * 16);
    }
  }
}

template <bool BLOCK, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void quantize_matrix_kernel(QuantizeArgs q) {
  quantize_tile<BLOCK, ROWS, COLS>(q, blockIdx.x);
}

// A product's gradients in one launch: dy both ways, x by its columns (Q'(x) of dw).
template <bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void quantize_gradients_kernel(QuantizeArgs dy, QuantizeArgs x) {
  const int t = blockIdx.x;
  if (t < dy.tiles) quantize_tile<false, ROWS, COLS>(dy, t);
  else quantize_tile<false, false, true>(x, t - dy.tiles);
}

static QuantizeArgs quantize_args(const void* x, int rows, int cols, void* out, void* out_t) {
  return QuantizeArgs{static_cast<const bf16_t*>(x), rows, cols, plan_fp8_mat(rows, cols), plan_fp8_mat(cols, rows),
                      static_cast<unsigned char*>(out), static_cast<unsigned char*>(out_t),
                      int(size_t((rows + 127) / 128) * ((cols + 127) / 128))};
}

hipError_t launch_quantize_matrix(const void* x, int rows, int cols, int block_rows, void* out, void* out_t,
                                  hipStream_t st) {
  const QuantizeArgs q = quantize_args(x, rows, cols, out, out_t);
  const dim3 grid(q.tiles), block(256);
#define LCM_Q(B, R, C) quantize_matrix_kernel<B, R, C><<<grid, block, 0, st>>>(q)
  if (block_rows == 128) {
    if (out && out_t) LCM_Q(true, true, true);
    else if (out) LCM_Q(true, true, false);
    else if (out_t) LCM_Q(true, false, true);
  } else {
    if (out && out_t) LCM_Q(false, true, true);
    else if (out) LCM_Q(false, true, false);
    else if (out_t) LCM_Q(false, false, true);
  }
#undef LCM_Q
  return hipGetLastError();
}

hipError_t launch_quantize_gradients(const void* dy, int T, int n, void* dyq, void* dyt, const void* x, int k, void* xt,
                                     hipStream_t st) {
  const QuantizeArgs a = quantize_args(dy, T, n, dyq, dyt), b = quantize_args(x, T, k, nullptr, xt);
  const dim3 grid(a.tiles + b.tiles), block(256);
  if (dyq) quantize_gradients_kernel<true, true><<<grid, block, 0, st>>>(a, b);
  else quantize_gradients_kernel<false, true><<<grid, block, 0, st>>>(a, b);
  return hipGetLastError();
}

}  // namespace lcm
