// Product of two block-FP8 matrices, C = A B^T (include/lc_moe_block.h).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies E4M3 codes and applies one E8M0 scale per row
// of A and of B and 32 reduction elements, taken from the lane that holds them.  The products
// are exact; the instruction adds its 64 products and the accumulator with about 12 bits below
// the largest addend.  The result's rounding to bf16 (8 bits) covers that but where the sum is much
// smaller than the root of its terms' squares: there the last bits of bf16 are the instruction's.
//
// A stage is 128 reduction columns, one scale block: BM + BN rows of 128 bytes, loaded into LDS
// directly, 16-byte piece c of row r in slot c ^ (r & 7) (eight lanes of a fragment read then
// fall on all banks), and the scale bytes of the tile's rows, laid out so that one word holds
// those of a lane's rows in four row blocks.
//
// Measured, products one after another (the card's clock moves with the length of the run: first 1 to 3 of
// them, then 30, then 300): 16384 x 6144 x 6144 in 535-550, 560, 500 us, 2.1-2.5 PFLOP/s of a dense peak near
// 5; 16384 x 6144 x 2048 in 196-216, 224, 190; 2048 x 6144 x 16384 in 189-201, 208, 179.  A library's FP8
// product with one scale a matrix, which has no scales to load, in the same runs: 402-427, 463, 400; 170-184,
// 187, 164; 159-178, 173, 151.  This tiling without the prefetched stream of stages took 690 where it took
// 500.  The matrix cores are busy 60% of the time.  A 256 x 256 tile is one wave per SIMD, so what a wave's
// reads of its fragments from LDS (128 KB a stage, half the time of the stage's products) and the barrier between
// stages do not hide stays: of a stage's 1.7 us, 1.4-1.6 remain without the loads from memory, 0.8 with the
// loads alone.  Tiles of 128 x 128, two a CU, read twice the bytes from the L2 (720 us where these take 580).
#include "block.h"
#include "lds_dma.h"
#include "train.h"

namespace lcm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Product {
  const unsigned char *a, *b;  // codes
  const unsigned char *as, *bs;
  size_t lda, ldb, las, lbs;
  const bf16_t* add;
  bf16_t* out;
  int M, N, nkb, chunk, splits, mt, nt;
};
struct MatmulArgs {
  Product p, q;  // the units of q follow those of p
  int units_p, units;
  float* part;
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
// has four neighbouring columns of one row.  TWO: the units of two products.
template <int MB, int NB, int MODE, bool TWO>
__global__ __launch_bounds__(256, MB == 4 ? 1 : 2) void matmul_fp8_kernel(MatmulArgs g) {
  constexpr int BM = MB * 64, BN = NB * 64;
  constexpr int ROWS = (BM + BN) * 128, STAGE = ROWS + 512;  // codes of A, of B, 256 scale bytes of each
  constexpr int LA = BM / 32, LB = BN / 32;                  // loads a wave and stage: 8 rows each
  constexpr int PER = LA + LB + 1;
  constexpr int NP = MB * NB;                                // products of a substep
  // Room of a wave for results on their way out: CB blocks of columns, 32 rows of them, or 16 where
  // two workgroups have to fit a CU.
  constexpr int CB = NB % 2 == 0 ? 2 : 1, OUT_ROWS = MB == 4 ? 32 : 16, OUT = OUT_ROWS * CB * 64;
  constexpr bool WHOLE_RUNS = BM % 128 == 0 && BN % 128 == 0;  // tiles start at a run of 128 scales
  __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * STAGE + 4 * OUT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, h = lane >> 5;

  // Every XCD takes a run of the units, in order: kGroup tiles of rows, then the columns, so that
  // the workgroups that run side by side on it share both operands in its L2.
  const int per_xcd = (g.units + 7) / 8;
  const int first = (blockIdx.x & 7) * per_xcd, last = min(first + per_xcd, g.units);
  const int step = int(gridDim.x >> 3);

#define LCM_OF(unit, field) (TWO && (unit) >= g.units_p ? g.q.field : g.p.field)
  struct Unit {
    int split, m0, n0, k0, nk;
  };
  auto unit_of = [&](int n) {
    Unit u;
    const int mt = LCM_OF(n, mt), nt = LCM_OF(n, nt), chunk = LCM_OF(n, chunk);
    const int in_product = TWO && n >= g.units_p ? n - g.units_p : n;
    u.split = in_product / (mt * nt);
    const int tile = in_product - u.split * (mt * nt);
    const int group = tile / (kGroup * nt), in = tile - group * (kGroup * nt);
    const int high = min(kGroup, mt - group * kGroup);
    u.n0 = in / high * BN;
    u.m0 = (group * kGroup + in % high) * BM;
    u.k0 = u.split * chunk;
    u.nk = min(chunk, LCM_OF(n, nkb) - u.k0);
    return u;
  };
  // The workgroup's stages are one stream through all its units; they are loaded two ahead.
  int ahead = first + int(blockIdx.x >> 3);  // unit of the next stage to load, and what is left of it
  if (ahead >= last) return;
  int unit = ahead, to_load = 0;
  const unsigned char *pa, *pb, *ps;  // the stage's rows and scales
  size_t sstep = 0;
  uint32_t off[LA + LB];  // the lane's pieces from there
  int runs = 0;           // where the tile's scales start in their runs: row blocks of A, of B << 8
  auto open = [&]() {
    const Unit u = unit_of(ahead);
    to_load = u.nk;
    const size_t lda = LCM_OF(ahead, lda), ldb = LCM_OF(ahead, ldb), las = LCM_OF(ahead, las), lbs = LCM_OF(ahead, lbs);
    pa = LCM_OF(ahead, a) + size_t(u.m0) * lda + size_t(u.k0) * 128;
    pb = LCM_OF(ahead, b) + size_t(u.n0) * ldb + size_t(u.k0) * 128;
    // scales: two waves load A's, two B's (the same bytes: one count for all waves)
    ps = (wave & 1) ? LCM_OF(ahead, bs) + size_t(u.k0) * lbs + (u.n0 & ~127)
                    : LCM_OF(ahead, as) + size_t(u.k0) * las + (u.m0 & ~127);
    sstep = (wave & 1) ? lbs : las;
    if constexpr (!WHOLE_RUNS) runs = (u.m0 >> 5 & 3) | (u.n0 >> 5 & 3) << 8;
    const int lane = here(tid) & 63, endA = LCM_OF(ahead, M) - u.m0 - 1, endB = LCM_OF(ahead, N) - u.n0 - 1;
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) {  // rows past the matrix read its last row and are not stored
      const bool isb = i >= LA;
      const int r = ((isb ? i - LA : i) * 4 + wave) * 8 + (lane >> 3);
      off[i] = uint32_t(min(r, isb ? endB : endA)) * uint32_t(isb ? ldb : lda) + (((lane & 7) ^ (r & 7)) << 4);
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
    ps = here(ps + by * sstep);
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
    else if (i < MB + NB) fa[ks][i - NB] = frag(st + (wm * MB + i - NB) * 32 * 128, ks);
  };
  // The scale bytes of the lane's rows in up to four row blocks from `block` of a run on: a word
  // holds those of four row blocks from a multiple of four on.
  auto scales = [&](const unsigned char* sc, int block, int count) {
    const unsigned char* w = sc + block / 4 * 128 + l32 * 4;
    const uint32_t lo = __builtin_bit_cast(uint32_t, *reinterpret_cast<const bf16x2*>(w));
    if (count != 3) return int(lo >> (block % 4 * 8));
    const uint32_t hi = __builtin_bit_cast(uint32_t, *reinterpret_cast<const bf16x2*>(w + 128));
    return int(__builtin_amdgcn_alignbyte(hi, lo, block % 4));
  };
  int sa, sb;
  auto read_scales = [&](const unsigned char* st, int runs) {
    sa = scales(st + ROWS, wm * MB + (WHOLE_RUNS ? 0 : runs & 0xFF), MB);
    sb = scales(st + ROWS + 256, wn * NB + (WHOLE_RUNS ? 0 : runs >> 8), NB);
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

  // Products of the first substep before the barrier behind which its stage's place is free, and
  // what goes beside each product: reads of operands, loads.
  constexpr int HALF = NP > 1 ? NP / 2 : 1, REST = NP - HALF;
  constexpr int READS = (MB + NB + HALF - 1) / HALF > 4 ? (MB + NB + HALF - 1) / HALF : 4;
  constexpr int EACH = REST > 0 ? (PER + REST - 1) / REST : PER;
  open();
  int runs0 = runs, runs1 = runs;  // of the stage at hand and the next
  for (int s = 0; s < 2; ++s) {
    runs1 = runs;
#pragma unroll
    for (int i = 0; i < PER; ++i) load_one(i, smem + s * STAGE);
    advance(by);
    if (--to_load == 0) next_load();
  }
  LCM_WAIT_VMCNT(PER);
  block_barrier();
#pragma unroll
  for (int i = 0; i < MB + NB; ++i) read_one(smem, 0, i);
  read_scales(smem, runs0);
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
        for (int i = k * READS; i < k * READS + READS; ++i) read_one(st, 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lds_reads();
      block_barrier();
#pragma unroll
      for (int k = 0; k < (REST > 0 ? REST : 1); ++k) {
        if (REST > 0) product(0, HALF + k, sa, sb);
#pragma unroll
        for (int i = k * EACH; i < k * EACH + EACH; ++i)
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
        constexpr int NEXT = NP >= 4 ? 4 : MB + NB;
#pragma unroll
        for (int i = k * NEXT; i < k * NEXT + NEXT; ++i) read_one(sn, 0, i);
        if (k == (NP > 2 ? 2 : 0)) read_scales(sn, runs1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!WHOLE_RUNS) runs1 = runs;
    }
    left -= n;
    to_load -= n;
    if (to_load == 0) next_load();
    if (left > 0) continue;
    const Unit done = unit_of(unit);
    // Lane: row l32 of a block, columns 8 (r / 4) + 4 h + r % 4.  Rows and columns past the matrix
    // are left out by the bounds of the buffer (32 rows of it).
    const int M = LCM_OF(unit, M), N = LCM_OF(unit, N);
    const int lane = here(tid) & 63, l32 = lane & 31, h = lane >> 5;
    unsigned char* room = smem + 2 * STAGE + wave * OUT;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row0 = done.m0 + (wm * MB + i) * 32, rows = max(min(M - row0, 32), 0);
      const size_t first = size_t(rows ? row0 : 0) * N;
      if constexpr (MODE == kPart) {
        const auto dst = buffer(g.part + size_t(done.split) * M * N + first, rows * N * 4);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          hold(acc[i][j]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = done.n0 + (wn * NB + j) * 32 + 8 * q + 4 * h;
            const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), dst,
                                                   col < N ? (l32 * N + col) * 4 : kNowhere, 0, 0);
          }
          zero(acc[i][j]);
        }
        continue;
      }
      // CB blocks of columns at a time through the wave's room: out in whole lines (CB = 2).  16-byte
      // piece c of row r is in a slot that spreads eight rows (CB = 1: sixteen) over the banks.
      auto slot_of = [](int r, int c) { return CB == 2 ? c ^ (r & 7) : c ^ (r >> 2 & 3); };
      const auto dst = buffer(LCM_OF(unit, out) + first, rows * N * 2);
      const auto add = buffer(MODE == kAdd ? LCM_OF(unit, add) + first : LCM_OF(unit, out), rows * N * 2);
#pragma unroll
      for (int jj = 0; jj < NB; jj += CB) {
        const int col0 = done.n0 + (wn * NB + jj) * 32;
        __builtin_amdgcn_sched_barrier(0);
        uint2 w[CB][4];
#pragma unroll
        for (int j = 0; j < CB; ++j) hold(acc[i][jj + j]);
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][jj + j][4 * q + e];
            if constexpr (MODE == kAdd) {
              const int col = col0 + j * 32 + 8 * q + 4 * h;
              const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(add, col < N ? (l32 * N + col) * 2 : kNowhere, 0, 0);
              v[0] += __uint_as_float(w[0] << 16), v[1] += __uint_as_float(w[0] & 0xFFFF0000u);
              v[2] += __uint_as_float(w[1] << 16), v[3] += __uint_as_float(w[1] & 0xFFFF0000u);
            }
            w[j][q] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
          }
#pragma unroll
        for (int j = 0; j < CB; ++j) zero(acc[i][jj + j]);
        constexpr int PIECES = CB * 4, AT_ONCE = 64 / PIECES;  // of a row; rows a store
        const int c = lane % PIECES, col = col0 + c * 8;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += OUT_ROWS) {
          if (OUT_ROWS == 32 || l32 / OUT_ROWS * OUT_ROWS == r0) {
            const int r = l32 % OUT_ROWS;
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint2*>(room + r * (CB * 64) + (slot_of(r, j * 4 + q) << 4) + h * 8) = w[j][q];
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int it = 0; it < OUT_ROWS / AT_ONCE; ++it) {
            const int r = it * AT_ONCE + lane / PIECES;
            const u32x4 w = *reinterpret_cast<const u32x4*>(room + r * (CB * 64) + (slot_of(r, c) << 4));
            __builtin_amdgcn_raw_buffer_store_b128(w, dst, col < N ? ((r0 + r) * N + col) * 2 : kNowhere, 0,
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
#undef LCM_OF
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

// Tiles of mb x nb times 64 x 64, and what they take (us, measured): a stage with 1 .. fit workgroups
// on a CU, and a unit's results.  In runs of 20, us in tiles of 256 x 256, 256 x 192, 128 x 128 and 64 x 64:
// M = 16384, N = K = 6144: 582, 632, 720, 1356; M = 2048, N = 6144, K = 16384 (192 tiles of the first, 256 of the
// second): 226, 205, 244, 386; M = 1024, N = 4096, K = 1536: 23.7, 20.8, 12.4, 15.7; M = N = K = 1000: 21.3, 15.6,
// 9.4, 6.7; M = 64, N = K = 6144: 23.5, 21.5, 16.1, 14.1.
struct Form {
  int mb, nb, fit;
  float stage[4], out;
};
constexpr Form kForms[] = {{4, 4, 1, {1.7f}, 1.5f},
                           {4, 3, 1, {1.3f}, 1.2f},
                           {2, 2, 2, {0.6f, 1.05f}, 0.5f},
                           {1, 1, 4, {0.35f, 0.5f, 0.7f, 0.92f}, 0.2f}};

MatmulPlan plan_matmul_fp8(int M, int N, int K) {
  MatmulPlan p{};
  const int nkb = (K + 127) / 128;
  // The form and the number of pieces of the reduction that take the least by these figures; pieces
  // are joined by a second kernel (2.5 us, their bytes at 5 TB/s): M = 64, N = K = 6144 takes 14 us in
  // four pieces, 20 in one.
  double best = 1e30;
  for (int f = 0; f < 4; ++f) {
    const Form& o = kForms[f];
    const size_t tiles = ((size_t(M) + o.mb * 64 - 1) / (o.mb * 64)) * ((size_t(N) + o.nb * 64 - 1) / (o.nb * 64));
    for (int want : {1, 2, 3, 4, 6, 8, 12, 16, 24}) {
      const int chunk = (nkb + want - 1) / want, splits = (nkb + chunk - 1) / chunk;
      if (splits != want || (splits > 1 && tiles * splits > 1024)) continue;
      const size_t each = (tiles * splits + 255) / 256;  // units of a CU
      double t = double(each / o.fit) * o.stage[o.fit - 1];
      if (each % o.fit) t += o.stage[each % o.fit - 1];
      t = 4 + t * chunk + o.out * each;
      if (splits > 1) t += 2.5 + double(splits) * M * N * 8 / 5e6;
      if (t < best) best = t, p.form = f, p.chunk = chunk;
    }
  }
  p.splits = (nkb + p.chunk - 1) / p.chunk;
  p.us = float(best);
  p.part = 0;
  p.total = p.splits > 1 ? align256(size_t(p.splits) * M * N * 4) : 256;
  return p;
}

static Product product_of(int M, int N, int K, const MatmulPlan& p, const void* a, const void* b, const void* add,
                          void* out) {
  const Fp8Mat am = plan_fp8_mat(M, K), bm = plan_fp8_mat(N, K);
  const unsigned char *ac = static_cast<const unsigned char*>(a), *bc = static_cast<const unsigned char*>(b);
  const int tm = kForms[p.form].mb * 64, tn = kForms[p.form].nb * 64;
  return Product{ac, bc, ac + am.scales, bc + bm.scales, am.ldc, bm.ldc, am.lds, bm.lds,
                 static_cast<const bf16_t*>(add), static_cast<bf16_t*>(out), M, N, am.nkb, p.chunk, p.splits,
                 (M + tm - 1) / tm, (N + tn - 1) / tn};
}

template <int MODE, bool TWO>
static void launch_form(int form, const MatmulArgs& g, hipStream_t st) {
  // as many workgroups as run at once, in whole rounds of the XCDs
  const int room = form <= 1 ? 256 : form == 2 ? 512 : 1024;
  const dim3 grid(unsigned(g.units < room ? (g.units + 7) / 8 * 8 : room)), block(256);
  switch (form) {
    case 0: if constexpr (!TWO) matmul_fp8_kernel<4, 4, MODE, TWO><<<grid, block, 0, st>>>(g); break;
    case 1: if constexpr (!TWO) matmul_fp8_kernel<4, 3, MODE, TWO><<<grid, block, 0, st>>>(g); break;
    case 2: matmul_fp8_kernel<2, 2, MODE, TWO><<<grid, block, 0, st>>>(g); break;
    default: matmul_fp8_kernel<1, 1, MODE, TWO><<<grid, block, 0, st>>>(g); break;
  }
}

hipError_t launch_matmul_join(const float* part, int splits, size_t n, const bf16_t* add, bf16_t* out, hipStream_t st) {
  matmul_join_kernel<<<dim3(unsigned((n / 8 + 255) / 256)), dim3(256), 0, st>>>(part, splits, n, add, out);
  return hipGetLastError();
}

hipError_t launch_matmul_fp8(int M, int N, int K, const MatmulPlan& p, void* ws, const void* a, const void* b,
                             const void* add, void* out, hipStream_t st) {
  MatmulArgs g{};
  g.p = product_of(M, N, K, p, a, b, add, out);
  g.units = g.units_p = g.p.mt * g.p.nt * p.splits;
  g.part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  if (g.part) launch_form<kPart, false>(p.form, g, st);
  else if (add) launch_form<kAdd, false>(p.form, g, st);
  else launch_form<kOut, false>(p.form, g, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_matmul_join(g.part, p.splits, size_t(M) * N, g.p.add, g.p.out, st);
}

hipError_t launch_matmul_gradients(int T, int k, int n, void* ws, const void* dyq, const void* w_t, const void* add,
                                   void* dx, const void* dyt, const void* xt, void* dw, hipStream_t st) {
  const MatmulPlan px = plan_matmul_fp8(T, k, n), pw = plan_matmul_fp8(n, k, T);
  // One launch instead of two (4 us of the host's time, and the second's start) for products that
  // leave the chip room: T = 777, k = 1032, n = 520.
  const bool one = px.form == pw.form && px.form >= 2 && px.splits == 1 && pw.splits == 1 && !add;
  if (!one) {
    const hipError_t e = launch_matmul_fp8(T, k, n, px, ws, dyq, w_t, add, dx, st);
    return e != hipSuccess ? e : launch_matmul_fp8(n, k, T, pw, ws, dyt, xt, nullptr, dw, st);
  }
  MatmulArgs g{};
  g.p = product_of(n, k, T, pw, dyt, xt, nullptr, dw);
  g.q = product_of(T, k, n, px, dyq, w_t, nullptr, dx);
  g.units_p = g.p.mt * g.p.nt;
  g.units = g.units_p + g.q.mt * g.q.nt;
  launch_form<kOut, true>(px.form, g, st);
  return hipGetLastError();
}

}  // namespace lcm
