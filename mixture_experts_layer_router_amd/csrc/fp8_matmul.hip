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
#include <type_traits>

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

// Keep a value out of the compiler's sight, in scalar or vector registers: what is made of it is made
// where it is used, not ahead of the loops, whose registers are all taken.
__device__ __forceinline__ const unsigned char* here(const unsigned char* p) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" : "+s"(p));
#endif
  return p;
}
__device__ __forceinline__ int here(int v) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(v));
#endif
  return v;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// What becomes of the sums: rounded, added to another matrix first, or kept as a piece in fp32.
enum { kOut, kAdd, kPart };
constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer below
// `bytes` (below 2^31) from p on; loads past them give 0, stores do nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);  // the same in every lane
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(a)), hi = __builtin_amdgcn_readfirstlane(uint32_t(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uint64_t(hi) << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr int kGroup = 4;  // tiles of rows that are taken together

// 2 x 2 waves; a wave holds MB x NB blocks of 32 x 32, as the transposes of C's blocks: a lane then
// has four neighbouring columns of one row.
template <int MB, int NB, int MODE>
__global__ __launch_bounds__(256, MB == 4 ? 1 : 2) void matmul_fp8_kernel(MatmulArgs p) {
  constexpr int BM = MB * 64, BN = NB * 64;
  constexpr int ROWS = (BM + BN) * 128, STAGE = ROWS + 512;  // codes of A, of B, 256 scale bytes of each
  constexpr int LA = BM / 32, LB = BN / 32;                  // loads a wave and stage: 8 rows each
  constexpr int PER = LA + LB + 1;
  constexpr int NP = MB * NB;                                // products of a substep
  // Room of a wave for results on their way out: 64 columns of 32 rows, of 16 where two workgroups
  // have to fit a CU.
  constexpr int OUT_ROWS = MB == 4 ? 32 : 16, OUT = OUT_ROWS * 128;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * STAGE + 4 * OUT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, h = lane >> 5;

  // Every XCD takes a run of the units, in order: kGroup tiles of rows, then the columns, so that
  // the workgroups that run side by side on it share both operands in its L2.
  const int tiles = p.mt * p.nt, units = tiles * p.splits, per_xcd = (units + 7) / 8;
  const int first = (blockIdx.x & 7) * per_xcd, last = min(first + per_xcd, units);
  const int step = int(gridDim.x >> 3);

  struct Unit {
    int split, m0, n0, k0, nk;
  };
  auto unit_of = [&](int unit) {
    Unit u;
    u.split = unit / tiles;
    const int tile = unit - u.split * tiles;
    const int group = tile / (kGroup * p.nt), in = tile - group * (kGroup * p.nt);
    const int high = min(kGroup, p.mt - group * kGroup);
    u.n0 = in / high * BN;
    u.m0 = (group * kGroup + in % high) * BM;
    u.k0 = u.split * p.chunk;
    u.nk = min(p.chunk, p.nkb - u.k0);
    return u;
  };
  // The workgroup's stages are one stream through all its units; they are loaded two ahead.
  int ahead = first + int(blockIdx.x >> 3);  // unit of the next stage to load, and what is left of it
  if (ahead >= last) return;
  int unit = ahead, to_load = 0;
  const unsigned char *pa, *pb, *ps;  // the stage's rows and scales
  uint32_t off[LA + LB];              // the lane's pieces from there
  auto open = [&]() {
    const Unit u = unit_of(ahead);
    to_load = u.nk;
    pa = p.a + size_t(u.m0) * p.lda + size_t(u.k0) * 128;
    pb = p.b + size_t(u.n0) * p.ldb + size_t(u.k0) * 128;
    // scales: two waves load A's, two B's (the same bytes: one count for all waves)
    ps = (wave & 1) ? p.bs + size_t(u.k0) * p.lbs + u.n0 : p.as + size_t(u.k0) * p.las + u.m0;
    const int lane = here(tid) & 63;
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) {  // rows past the matrix read its last row and are not stored
      const bool isb = i >= LA;
      const int r = ((isb ? i - LA : i) * 4 + wave) * 8 + (lane >> 3);
      const int end = (isb ? p.N - u.n0 : p.M - u.m0) - 1;
      off[i] = uint32_t(min(r, end)) * uint32_t(isb ? p.ldb : p.lda) + (((lane & 7) ^ (r & 7)) << 4);
    }
  };
  auto load_one = [&](int i, unsigned char* st) {
    if (i < LA)
      dma16(pa + off[i], st + (i * 4 + wave) * 1024);
    else if (i < LA + LB)
      dma16(pb + off[i], st + BM * 128 + ((i - LA) * 4 + wave) * 1024);
    else
      __builtin_amdgcn_global_load_lds(ps + uint32_t(lane * 4), (lds_void*)(st + ROWS + (wave & 1) * 256), 4, 0, 0);
  };
  // To the next stage of the same unit, by 0 or 1.
  auto advance = [&](int by) {
    pa = here(pa + by * 128);
    pb = here(pb + by * 128);
    ps = here(ps + by * ((wave & 1) ? p.lbs : p.las));
  };
  // Behind the last stage of a unit: the next unit.  Behind the last of all it stays there: the loads
  // that nobody needs keep a wave's count of loads the same in every stage.
  int by = 1;
  auto next_load = [&]() {
    ahead += step;
    if (ahead < last) {
      open();
      return;
    }
    advance(-by);
    by = 0;
    to_load = 1 << 30;
  };

  // LDS reads are of bf16 vectors throughout: reads of other types wait for every load in flight.
  // Piece c of row r is in slot c ^ (r & 7): the same swizzle in every row block.
  int at[2][2];  // byte offset of the lane's two pieces of a substep within a row block
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < 2; ++i) at[ks][i] = l32 * 128 + (((ks * 4 + h * 2 + i) ^ (l32 & 7)) << 4);
  auto frag = [&](const unsigned char* rows, int ks) {
    const i32x4 lo = __builtin_bit_cast(i32x4, *reinterpret_cast<const bf16x8*>(rows + at[ks][0]));
    const i32x4 hi = __builtin_bit_cast(i32x4, *reinterpret_cast<const bf16x8*>(rows + at[ks][1]));
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  i32x8 fa[2][MB], fb[2][NB];
  auto read_one = [&](const unsigned char* st, int ks, int i) {
    if (i < NB) fb[ks][i] = frag(st + (BM + (wn * NB + i) * 32) * 128, ks);
    else fa[ks][i - NB] = frag(st + (wm * MB + i - NB) * 32 * 128, ks);
  };
  // The scale bytes of the lane's rows in four row blocks of the tile: one word.  A wave of two
  // blocks shifts its own down.
  auto scales = [&](const unsigned char* sc, int block) {
    const uint32_t w = __builtin_bit_cast(uint32_t, *reinterpret_cast<const bf16x2*>(sc + block / 4 * 128 + l32 * 4));
    return int(w >> (block % 4 * 8));
  };
  f32x16 acc[MB][NB];
  auto product = [&](int ks, int k, int sa, int sb) {
    const int i = k / NB, j = k % NB;
#define LCM_MFMA(x, y) acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[ks][j], fa[ks][i], acc[i][j], 0, 0, y, sb, x, sa)
#define LCM_ROW(x) j == 0 ? LCM_MFMA(x, 0) : j == 1 ? LCM_MFMA(x, 1) : j == 2 ? LCM_MFMA(x, 2) : LCM_MFMA(x, 3)
    i == 0 ? LCM_ROW(0) : i == 1 ? LCM_ROW(1) : i == 2 ? LCM_ROW(2) : LCM_ROW(3);
#undef LCM_ROW
#undef LCM_MFMA
  };

  // Holds a sum in the accumulation registers at this point: left alone, the compiler fetches a
  // unit's sums all at once, and has no registers for them.
  auto hold = [&](f32x16& c) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+a"(c));
#endif
  };
  auto zero = [&](f32x16& c) {
#pragma unroll
    for (int r = 0; r < 16; ++r) c[r] = 0.f;
    hold(c);
  };
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) zero(acc[i][j]);

  constexpr int HALF = NP / 2, EACH = (PER + NP - HALF - 1) / (NP - HALF);
  open();
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load_one(i, smem + s * STAGE);
    advance(by);
    if (--to_load == 0) next_load();
  }
  LCM_WAIT_VMCNT(PER);
  block_barrier();
#pragma unroll
  for (int i = 0; i < MB + NB; ++i) read_one(smem, 0, i);
  int sa = scales(smem + ROWS, wm * MB), sb = scales(smem + ROWS + 256, wn * NB);
  int slot = 0, left = unit_of(unit).nk;
  while (true) {
    // The stages up to the end of a unit, of this one or of the one that is being loaded.
    const int n = min(left, to_load);
    for (int i = 0; i < n; ++i) {
      // A stage of two substeps.  Its second substep's operands are read beside the first's
      // products; once they are in registers (barrier) the stage after the next can be loaded into
      // its place, beside the rest of them; once the next stage has landed (no more loads in flight
      // than that one's; barrier) its first substep's operands are read beside the second's products.
      unsigned char* st = smem + slot * STAGE;
      slot ^= 1;
      const unsigned char* sn = smem + slot * STAGE;
      wait_lds_reads();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < HALF; ++k) {
        product(0, k, sa, sb);
#pragma unroll
        for (int i = k * 4; i < k * 4 + 4; ++i)
          if (i < MB + NB) read_one(st, 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds_reads();
      block_barrier();
#pragma unroll
      for (int k = HALF; k < NP; ++k) {
        product(0, k, sa, sb);
#pragma unroll
        for (int i = (k - HALF) * EACH; i < (k - HALF) * EACH + EACH; ++i)
          if (i < PER) load_one(i, st);
        __builtin_amdgcn_sched_barrier(0);
      }
      advance(by);
      LCM_WAIT_VMCNT(PER);
      block_barrier();
      const int ca = sa, cb = sb;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < NP; ++k) {  // (behind the last stage of all the reads find an old one: not used)
        product(1, k, ca, cb);
#pragma unroll
        for (int i = k * 4; i < k * 4 + 4; ++i)
          if (i < MB + NB) read_one(sn, 0, i);
        if (k == 2) sa = scales(sn + ROWS, wm * MB), sb = scales(sn + ROWS + 256, wn * NB);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    left -= n;
    to_load -= n;
    if (to_load == 0) next_load();
    if (left > 0) continue;
    const Unit done = unit_of(unit);
    // Lane: row l32 of a block, columns 8 (r / 4) + 4 h + r % 4.  Rows and columns past the matrix
    // are left out by the bounds of the buffer (32 rows of it), so that every unit stores as often.
    const int lane = here(tid) & 63, l32 = lane & 31, h = lane >> 5;
    unsigned char* room = smem + 2 * STAGE + wave * OUT;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row0 = done.m0 + (wm * MB + i) * 32, rows = max(min(p.M - row0, 32), 0);
      const size_t first = size_t(rows ? row0 : 0) * p.N;
      if constexpr (MODE == kPart) {
        const auto dst = buffer(p.part + size_t(done.split) * p.M * p.N + first, rows * p.N * 4);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          hold(acc[i][j]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = done.n0 + (wn * NB + j) * 32 + 8 * q + 4 * h;
            const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), dst,
                                                   col < p.N ? (l32 * p.N + col) * 4 : kNowhere, 0, 0);
          }
          zero(acc[i][j]);
        }
        continue;
      }
      // 64 columns at a time through the wave's room: out in whole lines.  16-byte piece c of row r is
      // in slot c ^ (r & 7).
      const auto dst = buffer(p.out + first, rows * p.N * 2);
      const auto add = buffer(MODE == kAdd ? p.add + first : p.out, rows * p.N * 2);
#pragma unroll
      for (int jj = 0; jj < NB; jj += 2) {
        const int col0 = done.n0 + (wn * NB + jj) * 32;
        __builtin_amdgcn_sched_barrier(0);
        hold(acc[i][jj]);
        hold(acc[i][jj + 1]);
        uint2 w[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][jj + j][4 * q + e];
            if constexpr (MODE == kAdd) {
              const int col = col0 + j * 32 + 8 * q + 4 * h;
              const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(add, col < p.N ? (l32 * p.N + col) * 2 : kNowhere, 0, 0);
              v[0] += __uint_as_float(w[0] << 16), v[1] += __uint_as_float(w[0] & 0xFFFF0000u);
              v[2] += __uint_as_float(w[1] << 16), v[3] += __uint_as_float(w[1] & 0xFFFF0000u);
            }
            w[j][q] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          }
        zero(acc[i][jj]);
        zero(acc[i][jj + 1]);
        const int c = lane & 7, col = col0 + c * 8;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += OUT_ROWS) {
          if (OUT_ROWS == 32 || l32 / OUT_ROWS * OUT_ROWS == r0) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2*>(room + l32 % OUT_ROWS * 128 + (((j * 4 + q) ^ (l32 & 7)) << 4) + h * 8) = w[j][q];
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int it = 0; it < OUT_ROWS / 8; ++it) {
            const int r = it * 8 + (lane >> 3);
            const u32x4 w = *reinterpret_cast<const u32x4*>(room + r * 128 + ((c ^ (r & 7)) << 4));
            __builtin_amdgcn_raw_buffer_store_b128(w, dst, col < p.N ? ((r0 + r) * p.N + col) * 2 : kNowhere, 0,
                                                   2);  // (streamed: nothing here reads it again)
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
      }
    }
    unit += step;
    if (unit >= last) break;
    left = unit_of(unit).nk;
  }
  LCM_WAIT_VMCNT(0);  // no load into this workgroup's LDS outlives it
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
  // as many workgroups as run at once, in whole rounds of the XCDs
  const size_t units = size_t(g.mt) * g.nt * p.splits, room = p.form == 0 ? 256 : 512;
  const unsigned grid = unsigned((units < room ? (units + 7) / 8 * 8 : room));
  const int mode = g.part ? kPart : add ? kAdd : kOut;
#define LCM_FORM(B)                                                                                   \
  do {                                                                                                \
    if (mode == kPart) matmul_fp8_kernel<B, B, kPart><<<dim3(grid), dim3(256), 0, st>>>(g);         \
    else if (mode == kAdd) matmul_fp8_kernel<B, B, kAdd><<<dim3(grid), dim3(256), 0, st>>>(g);      \
    else matmul_fp8_kernel<B, B, kOut><<<dim3(grid), dim3(256), 0, st>>>(g);                        \
  } while (0)
  if (p.form == 0) LCM_FORM(4);
  else LCM_FORM(2);
#undef LCM_FORM
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const size_t n = size_t(M) * N;
  matmul_join_kernel<<<dim3(unsigned((n / 8 + 255) / 256)), dim3(256), 0, st>>>(g.part, p.splits, n, g.add, g.out);
  return hipGetLastError();
}

}  // namespace lcm
