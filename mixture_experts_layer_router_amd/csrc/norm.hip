// Norms before and after a block with its gate and the scaled residual, and their gradient
// (include/lc_moe_block.h).
//
// A workgroup holds a row in registers, NV vectors of 16 bytes a thread, so every array of
// tokens is read and written once; the row's sums go through one barrier each.  It takes
// rows in turn, and keeps the weights (and, backward, its sums over tokens) in registers.
// Memory bounds both: bf16 T = 16384, d = 6144 takes 148 us forward (5.4 TB/s of four arrays) and 225
// backward (5.4 of six).
#include "block.h"
#include "topk.h"
#include "train.h"

namespace lcm {

template <typename E>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<bf16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void open(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 close(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void open(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 close(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

constexpr int kNormMaxThreads = 1024;

// Sums of C values over the workgroup, the same bits in every thread.  lds: two rooms used in
// turn, so that one barrier is enough: a room is written again only behind the next sum's
// barrier, which every thread reaches after it has read this one.  Waves that are not there have
// zeros in it (clear_sums).
constexpr int kMaxWaves = kNormMaxThreads / 64;
typedef float SumRoom[3][kMaxWaves];
__device__ __forceinline__ void clear_sums(SumRoom (&lds)[2]) {
  if (threadIdx.x < 2 * 3 * kMaxWaves) (&lds[0][0][0])[threadIdx.x] = 0.f;  // (a workgroup has 64 threads at least)
  if (threadIdx.x < 2 * 3 * kMaxWaves - 64) (&lds[0][0][0])[threadIdx.x + 64] = 0.f;
  __syncthreads();
}
template <int C>
__device__ __forceinline__ void block_sums(float (&v)[C], SumRoom (&lds)[2], int& turn) {
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = __ockl_wfred_add_f32(v[c]);
  if (blockDim.x == 64) return;
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  SumRoom& room = lds[turn];
  turn ^= 1;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) room[c][wave] = v[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    v[c] = 0.f;
    for (int w = 0; w < waves; w += 4) {
      const float4 q = *reinterpret_cast<const float4*>(&room[c][w]);
      v[c] += (q.x + q.y) + (q.z + q.w);
    }
  }
}

// Keeps a value out of the compiler's sight: what is made of it (addresses, the floats of a row) is made
// where it is used and not kept from one use for the next, nor ahead of the loop over rows.
__device__ __forceinline__ int here(int v) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(v));
#endif
  return v;
}
__device__ __forceinline__ uint4 here(uint4 v) {
  return make_uint4(here(int(v.x)), here(int(v.y)), here(int(v.z)), here(int(v.w)));
}

// The weights of vector j of thread tid, `other` without w and behind d.
template <typename E>
__device__ __forceinline__ void load_weight(const float* w, int tid, int j, int d, float other,
                                            float (&out)[Vec<E>::N]) {
  constexpr int N = Vec<E>::N;
  const int c = (tid + j * int(blockDim.x)) * N;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float4 q = make_float4(other, other, other, other);
    if (w && c < d) q = *reinterpret_cast<const float4*>(w + c + i);
    out[i] = q.x, out[i + 1] = q.y, out[i + 2] = q.z, out[i + 3] = q.w;
  }
}
template <typename E, int NV>
__device__ __forceinline__ void load_weights(const float* w, int d, float other, float (&out)[NV][Vec<E>::N]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) load_weight<E>(w, threadIdx.x, j, d, other, out[j]);
}

template <typename E, int NV>
__device__ __forceinline__ void load_rows(const void* p, size_t t, int d, int tid, uint4 (&out)[NV]) {
  constexpr int N = Vec<E>::N;
  const E* row = static_cast<const E*>(p) + t * d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (tid + j * int(blockDim.x)) * N;
    out[j] = p && c < d ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
  }
}

struct NormArgs {
  const void *x, *y;
  const float *gate, *w_post, *w_pre;
  void *h, *z;
  int T, d, gate_kind;
  float a, b, eps, rd;  // rd: 1 / d
};

template <typename E, int NV>
__global__ __launch_bounds__(kNormMaxThreads) void block_norm_kernel(NormArgs p) {
  constexpr int N = Vec<E>::N;
  __shared__ __attribute__((aligned(16))) SumRoom lds[2];
  int turn = 0;
  clear_sums(lds);
  float wpost[NV][N], wpre[NV][N], gc[NV][N];
  load_weights<E, NV>(p.w_post, p.d, 1.f, wpost);
  load_weights<E, NV>(p.w_pre, p.d, 0.f, wpre);
  load_weights<E, NV>(p.gate_kind == LC_MOE_GATE_CHANNEL ? p.gate : nullptr, p.d, 1.f, gc);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    uint4 qx[NV], qy[NV];
    load_rows<E, NV>(p.x, t, p.d, threadIdx.x, qx);
    load_rows<E, NV>(p.y, t, p.d, threadIdx.x, qy);
    float g = p.b;
    if (p.gate_kind == LC_MOE_GATE_TOKEN) g *= p.gate[t];
    float h[NV][N], s[1] = {0.f};
    if (p.w_post) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Vec<E>::open(qy[j], h[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] = fmaf(h[j][i], h[j][i], s[0]);
      }
      block_sums<1>(s, lds, turn);
      g *= 1.f / sqrtf(fmaf(s[0], p.rd, p.eps));
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[N], y[N];
      Vec<E>::open(qx[j], x);
      Vec<E>::open(qy[j], y);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        h[j][i] = fmaf(p.a, x[i], g * (y[i] * (wpost[j][i] * gc[j][i])));
        s[0] = fmaf(h[j][i], h[j][i], s[0]);
      }
    }
    if (p.z) {
      block_sums<1>(s, lds, turn);
      s[0] = 1.f / sqrtf(fmaf(s[0], p.rd, p.eps));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (int(threadIdx.x) + j * int(blockDim.x)) * N;
      if (c >= p.d) continue;
      const size_t at = size_t(t) * p.d + c;
      if (p.h) *reinterpret_cast<uint4*>(static_cast<E*>(p.h) + at) = Vec<E>::close(h[j]);
      if (p.z) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[j][i] *= s[0] * wpre[j][i];
        *reinterpret_cast<uint4*>(static_cast<E*>(p.z) + at) = Vec<E>::close(h[j]);
      }
    }
  }
}

// Threads of a row and vectors a thread: as few threads idle as may be.
static void norm_shape(int d, int vec, int& threads, int& nv) {
  const int n = (d + vec - 1) / vec;
  nv = 1;
  while ((n + nv - 1) / nv > kNormMaxThreads) ++nv;
  threads = ((n + nv - 1) / nv + 63) / 64 * 64;
}

template <typename E>
static hipError_t norm_forward(const NormArgs& p, hipStream_t st) {
  int threads, nv;
  norm_shape(p.d, Vec<E>::N, threads, nv);
  const int wgs = 256 * (2048 / threads);
  const dim3 grid(p.T < wgs ? p.T : wgs), block(threads);
  if (nv == 1) block_norm_kernel<E, 1><<<grid, block, 0, st>>>(p);
  else if (nv == 2) block_norm_kernel<E, 2><<<grid, block, 0, st>>>(p);
  else if constexpr (Vec<E>::N == 4) {  // (8 elements a vector: never more than two)
    if (nv == 3) block_norm_kernel<E, 3><<<grid, block, 0, st>>>(p);
    else block_norm_kernel<E, 4><<<grid, block, 0, st>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_block_norm(int T, int d, int dtype, const lc_moe_norm& n, const void* x, const void* y,
                             const float* gate, const float* w_post, const float* w_pre, void* h, void* z,
                             hipStream_t st) {
  const NormArgs p{x, y, gate, w_post, w_pre, h, z, T, d, n.gate_kind, n.residual_scale, n.block_scale, n.eps,
                   1.f / float(d)};
  return dtype == LC_MOE_BF16 ? norm_forward<bf16_t>(p, st) : norm_forward<float>(p, st);
}

// ---- gradient ----------------------------------------------------------------------------

struct NormBwArgs {
  const void *h, *dh, *dz, *y;
  const float *gate, *w_post, *w_pre;
  void *dx, *dy;
  float *part, *dgate_token;
  int T, d, gate_kind;
  float a, b, eps, rd;
};

// NEXT: the next row is loaded beside the present one's sums.  KEEP: the weights and all sums over tokens
// stay in registers; else the weights are read in every row again, from the L2, and two of the sums stay
// in LDS.  (With everything in registers, and spilled, d = 16384 ran at 1.3 TB/s; with these 3.9, 8192 rows in
// 410 us, fp32 4.8.)
template <typename E, int NV, int THREADS, bool NEXT, bool KEEP>
__global__ __launch_bounds__(THREADS) void block_norm_backward_kernel(NormBwArgs p) {
  constexpr int N = Vec<E>::N;
  __shared__ __attribute__((aligned(16))) SumRoom lds[2];
  __shared__ float4 room[!KEEP ? 2 : 1][!KEEP ? NV * N / 4 : 1][!KEEP ? THREADS : 1];
  int turn = 0;
  clear_sums(lds);
  float wpost[NV][N], wpre[NV][N], gc[NV][N];
  const float* wgate = p.gate_kind == LC_MOE_GATE_CHANNEL ? p.gate : nullptr;
  if (KEEP) {
    load_weights<E, NV>(p.w_post, p.d, 1.f, wpost);
    load_weights<E, NV>(p.w_pre, p.d, 0.f, wpre);
    load_weights<E, NV>(wgate, p.d, 1.f, gc);
  }
  float s_pre[NV][N], s_post[NV][N], s_gate[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s_pre[j][i] = s_post[j][i] = s_gate[j][i] = 0.f;
      if constexpr (!KEEP)
        room[0][(j * N + i) / 4][threadIdx.x] = room[1][(j * N + i) / 4][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  int tid = threadIdx.x;
  auto from_room = [&](int j) {
#pragma unroll
    for (int i = 0; i < N && !KEEP; i += 4) {
      const float4 f = room[0][(j * N + i) / 4][tid], g = room[1][(j * N + i) / 4][tid];
      s_post[j][i] = f.x, s_post[j][i + 1] = f.y, s_post[j][i + 2] = f.z, s_post[j][i + 3] = f.w;
      s_gate[j][i] = g.x, s_gate[j][i + 1] = g.y, s_gate[j][i + 2] = g.z, s_gate[j][i + 3] = g.w;
    }
  };
  auto to_room = [&](int j) {
#pragma unroll
    for (int i = 0; i < N && !KEEP; i += 4) {
      room[0][(j * N + i) / 4][tid] = make_float4(s_post[j][i], s_post[j][i + 1], s_post[j][i + 2], s_post[j][i + 3]);
      room[1][(j * N + i) / 4][tid] = make_float4(s_gate[j][i], s_gate[j][i + 1], s_gate[j][i + 2], s_gate[j][i + 3]);
    }
  };
  uint4 nh[NV], nd[NV], nz[NV], ny[NV];
  auto load = [&](int t) {
    if (!KEEP) tid = here(tid);
    load_rows<E, NV>(p.h, t, p.d, tid, nh);
    load_rows<E, NV>(p.dz, t, p.d, tid, nz);
    load_rows<E, NV>(p.y, t, p.d, tid, ny);
    load_rows<E, NV>(p.dh, t, p.d, tid, nd);
  };
  if (NEXT && blockIdx.x < p.T) load(blockIdx.x);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    if (!NEXT) load(t);
    uint4 qh[NV], qd[NV], qz[NV], qy[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) qh[j] = nh[j], qd[j] = nd[j], qz[j] = nz[j], qy[j] = ny[j];
    if (NEXT && p.T - t > int(gridDim.x)) load(t + gridDim.x);
    float g = p.b;
    if (p.gate_kind == LC_MOE_GATE_TOKEN) g *= p.gate[t];
    float s[3] = {0.f, 0.f, 0.f};  // h^2, w_pre dz h, y^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float h[N], z[N], y[N];
      if (!KEEP) tid = here(tid);
      Vec<E>::open(qh[j], h);
      Vec<E>::open(qz[j], z);
      Vec<E>::open(qy[j], y);
      if (!KEEP) load_weight<E>(p.w_pre, tid, j, p.d, 0.f, wpre[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[0] = fmaf(h[i], h[i], s[0]);
        s[1] = fmaf(wpre[j][i] * z[i], h[i], s[1]);
        s[2] = fmaf(y[i], y[i], s[2]);
      }
      if (!KEEP) __builtin_amdgcn_sched_barrier(0);
    }
    block_sums<3>(s, lds, turn);
    const float r = 1.f / sqrtf(fmaf(s[0], p.rd, p.eps));
    const float q = p.w_post ? 1.f / sqrtf(fmaf(s[2], p.rd, p.eps)) : 1.f;
    const float back = s[1] * p.rd * r * r;
    float dH[NV][N];
    float u[1] = {0.f};  // w_post y q gate dH, the token's gate left out
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float h[N], z[N], y[N], d[N];
      if (!KEEP) tid = here(tid), qh[j] = here(qh[j]), qz[j] = here(qz[j]), qy[j] = here(qy[j]);
      Vec<E>::open(qh[j], h);
      Vec<E>::open(qz[j], z);
      Vec<E>::open(qy[j], y);
      Vec<E>::open(qd[j], d);
      if (!KEEP) {
        load_weight<E>(p.w_pre, tid, j, p.d, 0.f, wpre[j]);
        load_weight<E>(p.w_post, tid, j, p.d, 1.f, wpost[j]);
        load_weight<E>(wgate, tid, j, p.d, 1.f, gc[j]);
      }
      if (!KEEP) from_room(j);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s_pre[j][i] = fmaf(z[i], h[i] * r, s_pre[j][i]);
        dH[j][i] = fmaf(r, wpre[j][i] * z[i] - h[i] * back, d[i]);
        const float yq = y[i] * q, wy = wpost[j][i] * yq;
        s_post[j][i] = fmaf(g * gc[j][i] * dH[j][i], yq, s_post[j][i]);
        s_gate[j][i] = fmaf(p.b * wy, dH[j][i], s_gate[j][i]);
        u[0] = fmaf(wy * gc[j][i], dH[j][i], u[0]);
      }
      if (!KEEP) to_room(j);
      if (!KEEP) __builtin_amdgcn_sched_barrier(0);
    }
    if (p.w_post || p.dgate_token) block_sums<1>(u, lds, turn);
    if (p.dgate_token && threadIdx.x == 0) p.dgate_token[t] = p.b * u[0];
    const float mean = g * u[0] * p.rd;  // of w_post du times y q
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!KEEP) tid = here(tid), qy[j] = here(qy[j]);
      const int c = (tid + j * int(blockDim.x)) * N;
      if (c >= p.d) continue;
      const size_t at = size_t(t) * p.d + c;
      if (p.dy) {
        float y[N];
        Vec<E>::open(qy[j], y);
        if (!KEEP) {
          load_weight<E>(p.w_post, tid, j, p.d, 1.f, wpost[j]);
          load_weight<E>(wgate, tid, j, p.d, 1.f, gc[j]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float du = g * gc[j][i] * dH[j][i];
          y[i] = p.w_post ? q * (wpost[j][i] * du - y[i] * q * mean) : du;
        }
        *reinterpret_cast<uint4*>(static_cast<E*>(p.dy) + at) = Vec<E>::close(y);
      }
      if (p.dx) {
#pragma unroll
        for (int i = 0; i < N; ++i) dH[j][i] *= p.a;
        *reinterpret_cast<uint4*>(static_cast<E*>(p.dx) + at) = Vec<E>::close(dH[j]);
      }
      if (!KEEP) __builtin_amdgcn_sched_barrier(0);
    }
  }
  float* part = p.part + size_t(blockIdx.x) * 3 * p.d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (int(threadIdx.x) + j * int(blockDim.x)) * N;
    if (c >= p.d) continue;
    if (!KEEP) from_room(j);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      *reinterpret_cast<float4*>(part + c + i) = make_float4(s_pre[j][i], s_pre[j][i + 1], s_pre[j][i + 2], s_pre[j][i + 3]);
      *reinterpret_cast<float4*>(part + p.d + c + i) =
          make_float4(s_post[j][i], s_post[j][i + 1], s_post[j][i + 2], s_post[j][i + 3]);
      *reinterpret_cast<float4*>(part + 2 * p.d + c + i) =
          make_float4(s_gate[j][i], s_gate[j][i + 1], s_gate[j][i + 2], s_gate[j][i + 3]);
    }
  }
}

// dst_k[c] = sum over the workgroups of part[w][k][c], in a fixed order: 64 columns a
// workgroup, its 16 waves a sixteenth of the rows each.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ part, int wgs, int d,
                                                         float* d0, float* d1, float* d2) {
  __shared__ float lds[16][64];
  float* dst = blockIdx.y == 0 ? d0 : blockIdx.y == 1 ? d1 : d2;
  if (!dst) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int w = wave; w < wgs; w += 16) s += part[(size_t(w) * 3 + blockIdx.y) * d + c];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += lds[w][lane];
    dst[c] = s;
  }
}

// One workgroup a CU takes rows in turn: at T = 16384, d = 6144 225 us with the next row on its way
// (5.4 TB/s), 270 without, 276 with two workgroups for each CU, which do not fit it at once; of up to 6
// waves two fit, of up to 3 four (T = 16384, d = 1032: 63 us with two of 3, 50 with four).  Beyond 256 of
// them a workgroup has two rows at least, or its sums over them are as many bytes as the rows (T = 600,
// d = 2048: 15.5 us with a row each, 13.6 with two).
// 8 elements a thread in up to 12 waves leave 168 registers (fp32, d = 6144: 315 us for 10922 tokens, 361
// with 16 elements in 6 waves), 16 in up to 8 waves 256, 16 in 16 waves 128: a row, and the sums in LDS.
struct NormBwShape {
  int threads, nv, per_cu;
};
static NormBwShape norm_backward_shape(int d, int vec) {
  const int n = (d + vec - 1) / vec, most = 16 / vec;  // vectors of a row, of a thread
  NormBwShape s{};
  s.nv = n <= 768 ? 1 : 2;
  while (s.nv < most && (n + s.nv - 1) / s.nv > 768) s.nv *= 2;
  s.threads = ((n + s.nv - 1) / s.nv + 63) / 64 * 64;
  s.per_cu = s.threads > 384 ? 1 : s.threads > 192 ? 2 : 4;
  return s;
}

NormBwPlan plan_norm_backward(int T, int d, int dtype) {
  NormBwPlan p{};
  int most = 256 * norm_backward_shape(d, dtype == LC_MOE_BF16 ? 8 : 4).per_cu;
  if (T / 2 < most) most = T / 2 < 256 ? 256 : T / 2;
  p.wgs = T < most ? T : most;
  p.part = 0;
  p.total = align256(size_t(p.wgs > 0 ? p.wgs : 1) * 3 * d * 4);
  return p;
}

template <typename E>
static void norm_backward(const NormBwArgs& p, int wgs, hipStream_t st) {
  const NormBwShape s = norm_backward_shape(p.d, Vec<E>::N);
  const dim3 grid(wgs), block(s.threads);
  constexpr int MOST = 16 / Vec<E>::N;
  if (s.nv == 1) block_norm_backward_kernel<E, 1, 768, true, true><<<grid, block, 0, st>>>(p);
  else if (s.nv == MOST && s.threads > 512)
    block_norm_backward_kernel<E, MOST, 1024, false, false><<<grid, block, 0, st>>>(p);
  else if (s.nv == MOST) block_norm_backward_kernel<E, MOST, 512, true, MOST == 2><<<grid, block, 0, st>>>(p);
  else if constexpr (MOST > 2) block_norm_backward_kernel<E, 2, 768, true, true><<<grid, block, 0, st>>>(p);
}

hipError_t launch_block_norm_backward(int T, int d, int dtype, const lc_moe_norm& n, const NormBwPlan& plan, void* ws,
                                      const void* h, const void* dh, const void* dz, const void* y,
                                      const float* gate, const float* w_post, const float* w_pre, void* dx, void* dy,
                                      float* dw_pre, float* dw_post, float* dgate, hipStream_t st) {
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.part);
  const bool token = n.gate_kind == LC_MOE_GATE_TOKEN;
  const NormBwArgs p{h, dh, dz, y, gate, w_post, w_pre, dx, dy, part, token ? dgate : nullptr, T, d, n.gate_kind,
                     n.residual_scale, n.block_scale, n.eps, 1.f / float(d)};
  if (plan.wgs > 0) {
    if (dtype == LC_MOE_BF16) norm_backward<bf16_t>(p, plan.wgs, st);
    else norm_backward<float>(p, plan.wgs, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  float* dg = token ? nullptr : dgate;
  if (dw_pre || dw_post || dg)
    norm_sums_kernel<<<dim3((d + 63) / 64, 3), dim3(1024), 0, st>>>(part, plan.wgs, d, dw_pre, dw_post, dg);
  return hipGetLastError();
}

}  // namespace lcm
