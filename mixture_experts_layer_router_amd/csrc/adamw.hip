// One AdamW step over many tensors (formulas and the form of the 8-bit states in
// include/lc_moe_train.h).  A step reads and writes every byte of the weights and states
// once: it is bound by HBM.  The tensors' addresses travel in the kernel's arguments, up to
// kMaxTensors a launch, so a step of a few dozen tensors is one launch and needs no device
// table.
#include <cmath>

#include "fp8.h"
#include "topk.h"
#include "train.h"

namespace lcm {

namespace aw {

constexpr int kMaxTensors = 32;  // descriptors per launch (kernel arguments stay below 4 KB)
constexpr int kChunk = 2048;     // elements per workgroup: 256 threads x 8

struct Desc {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  int64_t n;
  float wd, lrs;
  int64_t at;      // first element of this launch's piece (a multiple of kChunk)
  uint32_t first;  // first workgroup of the piece
  uint32_t flags;  // 1: param bf16, 2: grad bf16; place in the caller's list << 2
};
struct Args {
  Desc t[kMaxTensors];
  int count;  // pieces of this launch
  float lr, beta1, omb1, beta2, omb2, eps;
  double ln1, ln2;  // log(beta1), log(beta2); -infinity for 0
  int step;
  const int32_t* step_dev;
  const float* grad_scale;
  uint32_t seed;
};
static_assert(sizeof(Args) <= 4000, "kernel arguments");

// a * b and a + b, each rounded by itself: the compiler may not join them into one
// multiply-add, so the states (and the codes taken from them) are the formula's to the bit.
__device__ __forceinline__ float mul(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}
__device__ __forceinline__ float add(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// 32-bit mixing: shifts that fold the high bits down and odd multipliers (the fractional
// digits of the square roots of 2 and 3)
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// E4M3 code of |y| <= 448 rounded down or up by the 20-bit fraction r: the digits below the
// code's last place plus r carry into it with probability (their size) / (one step).
__device__ __forceinline__ uint32_t e4m3_random(float y, uint32_t r) {
  const float a = fabsf(y);
  uint32_t q;
  if (a < 0.015625f) q = static_cast<uint32_t>(add(a * 512.f, static_cast<float>(r) * 9.5367431640625e-07f));
  else q = ((__float_as_uint(a) + r) >> 20) - 960u;
  q = q < 126u ? q : 126u;
  return q | (y < 0.f ? 128u : 0u);
}

// Value of an E4M3 code (finite codes only).
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t e = (c >> 3) & 15u, f = c & 7u;
  const float a = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : static_cast<float>(f) * 0.001953125f;
  return c & 128u ? -a : a;
}

__device__ __forceinline__ float pow2(int k) {  // 2^k, k in -127..127
  return k >= -126 ? __uint_as_float(uint32_t(k + 127) << 23) : __uint_as_float(1u << 22);
}

// 8 elements of a tensor as fp32; cnt < 8 only at its end.
__device__ __forceinline__ void load8(const void* p, bool bf, int64_t i, int cnt, float (&o)[8]) {
  if (bf) {
    const bf16_t* q = static_cast<const bf16_t*>(p) + i;
    if (cnt == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(q);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[2 * c] = __uint_as_float(u[c] << 16);
        o[2 * c + 1] = __uint_as_float(u[c] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = c < cnt ? bf2f(q[c]) : 0.f;
    }
  } else {
    const float* q = static_cast<const float*>(p) + i;
    if (cnt == 8) {
      const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
      o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = c < cnt ? q[c] : 0.f;
    }
  }
}
__device__ __forceinline__ void store8(void* p, bool bf, int64_t i, int cnt, const float (&o)[8]) {
  if (bf) {
    bf16_t* q = static_cast<bf16_t*>(p) + i;
    if (cnt == 8) {
      uint32_t u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) u[c] = f2bf(o[2 * c]) | (uint32_t(f2bf(o[2 * c + 1])) << 16);
      *reinterpret_cast<uint4*>(q) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cnt) q[c] = f2bf(o[c]);
    }
  } else {
    float* q = static_cast<float*>(p) + i;
    if (cnt == 8) {
      *reinterpret_cast<float4*>(q) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(o[4], o[5], o[6], o[7]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cnt) q[c] = o[c];
    }
  }
}

__device__ __forceinline__ uint2 load_codes(const void* p, int64_t i, int cnt) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + i;
  if (cnt == 8) return *reinterpret_cast<const uint2*>(q);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < cnt) w[c >> 2] |= uint32_t(q[c]) << (8 * (c & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int cnt, uint2 v) {
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if (cnt == 8) {
    *reinterpret_cast<uint2*>(q) = v;
    return;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < cnt) q[c] = uint8_t((c < 4 ? v.x : v.y) >> (8 * (c & 3)));
}

// Block exponent (at least -127) of 16 lanes x 8 values.
__device__ __forceinline__ int block_k(const float (&val)[8]) {
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(val[c]));
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
  const int k = block_exp(amax);
  return k < -127 ? -127 : k;
}

}  // namespace aw

template <int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(aw::Args a) {
  using namespace aw;
  // 8 bits: 2^-k of every exponent byte, from the math library's powf.  It may be an ulp off
  // the power of two, 2^-20 of a code's step; tensor libraries scale by it too, so the codes
  // equal those of a program that computes the step with elementary tensor operations.
  __shared__ float inverse[BITS == 8 ? 256 : 1];
  if constexpr (BITS == 8) {
    inverse[threadIdx.x] = powf(2.f, 127.f - static_cast<float>(threadIdx.x));
    __syncthreads();
  }
  int ti = 0;
  for (int i = 1; i < a.count; ++i) ti = a.t[i].first <= blockIdx.x ? i : ti;
  const Desc& t = a.t[ti];
  float gs = 1.f;
  if (a.grad_scale) {
    gs = *a.grad_scale;
    if (!(fabsf(gs) < INFINITY)) return;
  }
  int step = a.step_dev ? *a.step_dev : a.step;
  step = step < 1 ? 1 : step;
  // 1 - beta^step = -expm1(step log beta)
  const float rate = static_cast<float>(double(a.lr) * t.lrs / -expm1(step * a.ln1));
  const float root = static_cast<float>(1. / sqrt(-expm1(step * a.ln2)));
  const float keep = static_cast<float>(1. - double(a.lr) * t.lrs * t.wd);
  const int64_t i = t.at + int64_t(blockIdx.x - t.first) * kChunk + threadIdx.x * 8;
  const int cnt = t.n - i >= 8 ? 8 : t.n > i ? int(t.n - i) : 0;
  float g[8], w[8], m[8], v[8], r[8];
  load8(t.grad, t.flags & 2, i, cnt, g);
  if (t.master) load8(t.master, false, i, cnt, w);
  else load8(t.param, t.flags & 1, i, cnt, w);
  if constexpr (BITS == 32) {
    load8(t.m, false, i, cnt, m);
    load8(t.v, false, i, cnt, v);
  } else {
    const uint2 cm = load_codes(t.m, i, cnt), cv = load_codes(t.v, i, cnt);
    const float sm = cnt ? pow2(int(t.ms[i >> 7]) - 127) : 0.f, sv = cnt ? pow2(int(t.vs[i >> 7]) - 127) : 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = e4m3_value(((c < 4 ? cm.x : cm.y) >> (8 * (c & 3))) & 255u) * sm;
      const float q = e4m3_value(((c < 4 ? cv.x : cv.y) >> (8 * (c & 3))) & 255u) * sv;
      v[c] = mul(q, q);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float gr = mul(g[c], gs);
    m[c] = add(mul(a.beta1, m[c]), mul(a.omb1, gr));
    v[c] = add(mul(a.beta2, v[c]), mul(mul(a.omb2, gr), gr));
    r[c] = sqrtf(v[c]);  // rounded to nearest (the default of this compiler)
    w[c] = w[c] * keep - rate * (m[c] / (r[c] * root + a.eps));
  }
  if (t.master) store8(t.master, false, i, cnt, w);
  store8(t.param, t.flags & 1, i, cnt, w);
  if constexpr (BITS == 32) {
    store8(t.m, false, i, cnt, m);
    store8(t.v, false, i, cnt, v);
  } else {
    const uint32_t key = mix(mix(a.seed + 0x9E3779B9u * uint32_t(step)) + 0x3C6EF373u * ((t.flags >> 2) + 1u) +
                             0x85A308D3u * uint32_t(uint64_t(i) >> 32));
    const int km = block_k(m), kv = block_k(r);
    const float im = inverse[km + 127], iv = inverse[kv + 127];
    uint32_t qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t u = mix(uint32_t(i) + c + key);
      qm[c >> 2] |= e4m3_random(m[c] * im, ((u & 0xFFFFu) << 4) + 8u) << (8 * (c & 3));
      uint32_t q = e4m3_random(r[c] * iv, ((u >> 16) << 4) + 8u);
      q = r[c] > 0.f && q == 0u ? 1u : q;
      qv[c >> 2] |= q << (8 * (c & 3));
    }
    store_codes(t.m, i, cnt, make_uint2(qm[0], qm[1]));
    store_codes(t.v, i, cnt, make_uint2(qv[0], qv[1]));
    if ((threadIdx.x & 15) == 0 && cnt) {
      t.ms[i >> 7] = uint8_t(km + 127);
      t.vs[i >> 7] = uint8_t(kv + 127);
    }
  }
}

hipError_t launch_adamw(const lc_moe_adamw_tensor* tensors, int count, const lc_moe_adamw_hyper& h, hipStream_t st) {
  using namespace aw;
  Args a{};
  a.lr = h.lr;
  a.beta1 = h.beta1;
  a.omb1 = static_cast<float>(1. - double(h.beta1));
  a.beta2 = h.beta2;
  a.omb2 = static_cast<float>(1. - double(h.beta2));
  a.eps = h.eps;
  a.ln1 = std::log(double(h.beta1));
  a.ln2 = std::log(double(h.beta2));
  a.step = h.step;
  a.step_dev = h.step_dev;
  a.grad_scale = h.grad_scale;
  a.seed = h.seed;
  // One launch covers up to kMaxTensors pieces and kMaxBlocks workgroups (the grid holds
  // 2^32 - 1 work-items); a tensor that needs more is cut at a multiple of its blocks.
  constexpr int64_t kMaxBlocks = int64_t(1) << 23;
  int64_t blocks = 0;
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    if (h.state_bits == 32) hipLaunchKernelGGL(adamw_kernel<32>, dim3(unsigned(blocks)), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(adamw_kernel<8>, dim3(unsigned(blocks)), dim3(256), 0, st, a);
    a.count = 0;
    blocks = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    const lc_moe_adamw_tensor& t = tensors[i];
    for (int64_t at = 0; at < t.n;) {
      if (a.count == kMaxTensors || blocks == kMaxBlocks) {
        const hipError_t err = flush();
        if (err != hipSuccess) return err;
      }
      int64_t take = (t.n - at + kChunk - 1) / kChunk;
      if (take > kMaxBlocks - blocks) take = kMaxBlocks - blocks;
      Desc& d = a.t[a.count++];
      d.param = t.param;
      d.master = t.master;
      d.grad = t.grad;
      d.m = t.m;
      d.v = t.v;
      d.ms = t.m_scale;
      d.vs = t.v_scale;
      d.n = t.n;
      d.wd = t.weight_decay;
      d.lrs = t.lr_scale;
      d.at = at;
      d.first = uint32_t(blocks);
      d.flags = (t.param_dtype == LC_MOE_BF16 ? 1u : 0u) | (t.grad_dtype == LC_MOE_BF16 ? 2u : 0u) | (uint32_t(i) << 2);
      blocks += take;
      at += take * kChunk;
    }
  }
  return flush();
}

}  // namespace lcm
