// One AdamW step over many tensors (formulas and the form of the 8-bit states in
// include/lc_moe_train.h).  A step reads and writes every byte of the weights and states
// once: it is bound by HBM.  403M bf16 weights with fp32 masters and 32-bit states (28 bytes a
// weight) take 2.13 ms, 5.3 TB/s, where a copy reaches 4.9.  With 8-bit states and no masters (10
// bytes) 0.77 ms, 5.2 TB/s: there the arithmetic (the hash, two random roundings, a root)
// counts beside the bytes.  Steps: 1.25 ms with codes decoded in integer arithmetic and
// 1 - beta^step by expm1 in every thread, 0.84 without, 0.795 with strips typed by what the
// tensors hold, 0.78 with the hardware's random rounding, which also takes the registers from 94
// to 67, 0.735 with one strip a workgroup instead of four; codes settled in fp64 where fp32 would
// decide them took it to 0.765 (80 registers; the fp64 values of every element, unrolled, 0.83).
// The tensors' addresses travel in the kernel's arguments, up to kMaxTensors a launch, so a
// step of a few dozen tensors is one launch and needs no device table.
#include <cmath>
#include <type_traits>

#include "fp8.h"
#include "topk.h"
#include "train.h"

namespace lcm {

namespace aw {

constexpr int kStrip = 2048;  // elements a workgroup takes at a time: 256 threads x 8

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
  uint32_t at;     // first strip of this launch's piece of the tensor
  uint32_t flags;  // 1: param bf16, 2: grad bf16; place in the caller's list << 2
};
struct Hyper {
  float lr, beta1, omb1, beta2, omb2, eps;
  double p1, p2;  // beta1^step, beta2^step
  uint32_t seed;
  int step;
  const int32_t* step_dev;
  const float* grad_scale;
};
// Descriptors per launch: as many as fit in 4000 bytes of kernel arguments with the first
// workgroup of each piece beside them.
constexpr int kMaxTensors = int((4000 - sizeof(Hyper) - 8) / (sizeof(Desc) + 4));
struct Args {
  Hyper h;
  int count;
  uint32_t first[kMaxTensors];
  Desc t[kMaxTensors];
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

// beta^t by squaring, products only: the same bits on the host and on the device.
__host__ __device__ inline double power(double b, int t) {
#pragma clang fp contract(off)
  double r = 1.;
  for (; t; t >>= 1) {
    if (t & 1) r = r * b;
    b = b * b;
  }
  return r;
}
// The step's scalars of a tensor: the rate over 1 - beta1^t, 1 / sqrt(1 - beta2^t), the decay.
struct Scalars {
  float rate, root, keep;
};
__device__ __forceinline__ Scalars scalars(const Hyper& h, float lrs, float wd, double p1, double p2) {
#pragma clang fp contract(off)
  const double lr = double(h.lr) * lrs;
  return Scalars{static_cast<float>(lr / (1. - p1)), static_cast<float>(1. / sqrt(1. - p2)),
                 static_cast<float>(1. - lr * wd)};
}

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

// The square root rounded to nearest for 2^-100 <= v < infinity: v / sqrt(v) from the
// hardware's reciprocal root (one ulp) and one correction by the exact residual, which leaves
// about 2^-46 before the last rounding.
__device__ __forceinline__ float root_of(float v) {
  const float y = __builtin_amdgcn_rsqf(v);
  const float s = v * y;
  return fmaf(fmaf(-s, s, v), 0.5f * y, s);
}

__device__ __forceinline__ float pow2(int k) {  // 2^k, k in -127..127
  return k >= -126 ? __uint_as_float(uint32_t(k + 127) << 23) : __uint_as_float(1u << 22);
}

// 4 elements of a tensor as fp32; cnt < 4 only at its end.
__device__ __forceinline__ void load4(const void* p, bool bf, int64_t i, int cnt, float* o) {
  if (bf) {
    const bf16_t* q = static_cast<const bf16_t*>(p) + i;
    if (cnt >= 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      o[0] = __uint_as_float(w.x << 16), o[1] = __uint_as_float(w.x & 0xFFFF0000u);
      o[2] = __uint_as_float(w.y << 16), o[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = c < cnt ? bf2f(q[c]) : 0.f;
    }
  } else {
    const float* q = static_cast<const float*>(p) + i;
    if (cnt >= 4) {
      const float4 a = *reinterpret_cast<const float4*>(q);
      o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = c < cnt ? q[c] : 0.f;
    }
  }
}
__device__ __forceinline__ void store4(void* p, bool bf, int64_t i, int cnt, const float* o) {
  if (bf) {
    bf16_t* q = static_cast<bf16_t*>(p) + i;
    if (cnt >= 4) {
      *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < cnt) q[c] = f2bf(o[c]);
    }
  } else {
    float* q = static_cast<float*>(p) + i;
    if (cnt >= 4) {
      *reinterpret_cast<float4*>(q) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < cnt) q[c] = o[c];
    }
  }
}
// A thread's 8 elements of a strip, in two groups of 4 that are GAP elements apart.
template <int GAP>
__device__ __forceinline__ void load8(const void* p, bool bf, int64_t i, const int (&cnt)[2], float (&o)[8]) {
  if (GAP == 4 && bf && cnt[1] == 4) {  // 16 bytes
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const bf16_t*>(p) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      o[2 * c] = __uint_as_float(u[c] << 16);
      o[2 * c + 1] = __uint_as_float(u[c] & 0xFFFF0000u);
    }
    return;
  }
  load4(p, bf, i, cnt[0], o);
  load4(p, bf, i + GAP, cnt[1], o + 4);
}
template <int GAP>
__device__ __forceinline__ void store8(void* p, bool bf, int64_t i, const int (&cnt)[2], const float (&o)[8]) {
  if (GAP == 4 && bf && cnt[1] == 4) {
    *reinterpret_cast<uint4*>(static_cast<bf16_t*>(p) + i) =
        make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
    return;
  }
  store4(p, bf, i, cnt[0], o);
  store4(p, bf, i + GAP, cnt[1], o + 4);
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

// The largest magnitude of a row of 16 lanes' values, from each lane's.
template <int CTRL>
__device__ __forceinline__ float row_max(float v) {
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 15, 15, true)));
}
__device__ __forceinline__ float block_max(const float (&val)[8]) {
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(val[c]));
  // rotations of the row by 8, 4, 2, 1 lanes
  return row_max<0x121>(row_max<0x122>(row_max<0x124>(row_max<0x128>(amax))));
}
// Exponent byte of a block: 2^(byte - 127) is the smallest power of two p with amax <= 448 p,
// at least 2^-127; 127 for zeros.  448 = 1.75 2^8, so a mantissa above 1.75 carries.
__device__ __forceinline__ int block_byte(float amax) {
  const uint32_t u = __float_as_uint(amax), k = (u + 0x1FFFFFu) >> 23;
  return u == 0u ? 127 : k > 8u ? int(k) - 8 : 0;
}

// 8 codes times their scale, two at a time (v_cvt_scalef32_pk_f32_fp8)
__device__ __forceinline__ void decode(uint2 q, float scale, float (&o)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const uint32_t u[2] = {q.x, q.y};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const f32x2 d = c & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(u[c >> 1], scale, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(u[c >> 1], scale, false);
    o[2 * c] = d[0], o[2 * c + 1] = d[1];
  }
}

// The random words of a value's two codes, 16 bits each and half a unit of them.
__device__ __forceinline__ uint32_t word_m(uint32_t u) { return (u << 16) | 0x8000u; }
__device__ __forceinline__ uint32_t word_v(uint32_t u) { return (u & 0xFFFF0000u) | 0x8000u; }

// E4M3 codes of 8 values y rounded down or up by chance (v_cvt_sr_fp8_f32): the digits below the
// code's last place plus the top 20 of the 32 random bits carry into it with probability
// (their size) / (one step); below 2^-6 the steps are 2^-9.
__device__ __forceinline__ void encode(const float (&m)[8], const float (&r)[8], const uint32_t (&u)[8], uint2& cm, uint2& cv) {
  int qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    qm[c] = __builtin_amdgcn_cvt_sr_fp8_f32(m[4 * c], word_m(u[4 * c]), qm[c], 0);
    qm[c] = __builtin_amdgcn_cvt_sr_fp8_f32(m[4 * c + 1], word_m(u[4 * c + 1]), qm[c], 1);
    qm[c] = __builtin_amdgcn_cvt_sr_fp8_f32(m[4 * c + 2], word_m(u[4 * c + 2]), qm[c], 2);
    qm[c] = __builtin_amdgcn_cvt_sr_fp8_f32(m[4 * c + 3], word_m(u[4 * c + 3]), qm[c], 3);
    qv[c] = __builtin_amdgcn_cvt_sr_fp8_f32(r[4 * c], word_v(u[4 * c]), qv[c], 0);
    qv[c] = __builtin_amdgcn_cvt_sr_fp8_f32(r[4 * c + 1], word_v(u[4 * c + 1]), qv[c], 1);
    qv[c] = __builtin_amdgcn_cvt_sr_fp8_f32(r[4 * c + 2], word_v(u[4 * c + 2]), qv[c], 2);
    qv[c] = __builtin_amdgcn_cvt_sr_fp8_f32(r[4 * c + 3], word_v(u[4 * c + 3]), qv[c], 3);
  }
  cm = make_uint2(qm[0], qm[1]);
  cv = make_uint2(qv[0], qv[1]);
}

// Steps of fp32 from the value at which the random word just carries up to y, in the top 20 bits
// (whole numbers modulo 2^20, as digits below the code's last place are).
__device__ __forceinline__ uint32_t past(float y, uint32_t word) { return (__float_as_uint(y) << 12) + word; }
// Whether y lies within two steps of that value; below 2^-6 codes have other borders.
__device__ __forceinline__ bool at_border(float y, uint32_t word) {
  return past(y, word) + 0x2000u <= 0x3000u && fabsf(y) >= 0.015625f && fabsf(y) <= 448.f;
}

}  // namespace aw

// One workgroup takes one strip of one tensor, so that the workgroups in flight touch neighbouring
// memory (403M weights: 32-bit states and masters 2109 us, 2126 with two strips, 2171 with four;
// 8-bit states 748, 778, 781).  A thread has 8 elements of it, with 8-bit states consecutive ones,
// a row of 16 lanes one block of the states.
template <int BITS>
__global__ __launch_bounds__(256, BITS == 8 ? 5 : 6) void adamw_kernel(aw::Args a) {
  using namespace aw;
  const Hyper& h = a.h;
  int ti = 0;
  for (int i = 1; i < a.count; ++i) ti = a.first[i] <= blockIdx.x ? i : ti;
  const Desc& t = a.t[ti];
  float gs = 1.f;
  if (h.grad_scale) gs = *h.grad_scale;
  // A scale that is not finite leaves the step out.  32 bits: asked for behind the strip's loads,
  // which it would hold up (40 small tensors: 9.7 us before, 7.2 behind); 8 bits: no difference for
  // 403M weights.
  const bool finite = fabsf(gs) < INFINITY;
  if (BITS == 8 && !finite) return;
  int step = h.step;
  double p1 = h.p1, p2 = h.p2;
  if (h.step_dev) {
    step = *h.step_dev;
    step = step < 1 ? 1 : step;
    p1 = power(double(h.beta1), step);
    p2 = power(double(h.beta2), step);
  }
  const Scalars sc = scalars(h, t.lrs, t.wd, p1, p2);
  const uint32_t key0 = mix(h.seed + 0x9E3779B9u * uint32_t(step)) + 0x3C6EF373u * ((t.flags >> 2) + 1u);
  const int64_t strip0 = int64_t(t.at) + int64_t(blockIdx.x - a.first[ti]);
  // 32 bits: groups of 4 with a strip's half between them, so that every load and store of
  // fp32 values is one contiguous piece of a wave; 8 bits: 8 consecutive elements
  constexpr int GAP = BITS == 32 ? kStrip / 2 : 4;
  const int mine = threadIdx.x * (BITS == 32 ? 4 : 8);  // the thread's place in a strip
  // The update of a thread's elements from i on (two: how many of each group) from their
  // gradients, weights and states (8 bits: codes cm, cv of scales sm, sv)
  auto update = [&](int64_t i, const int (&two)[2], const float (&g)[8], float (&w)[8], float (&m)[8], float (&v)[8],
                    uint2 cm, uint2 cv, float sm, float sv) {
    const int cnt = two[0] + two[1];
    float r[8];
    if constexpr (BITS == 8) {
      decode(cm, sm, m);
      decode(cv, sv, r);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = mul(r[c], r[c]);
    }
    if (BITS == 32 && !finite) return;
    float least = INFINITY, most = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float gr = mul(g[c], gs);
      m[c] = add(mul(h.beta1, m[c]), mul(h.omb1, gr));
      v[c] = add(mul(h.beta2, v[c]), mul(mul(h.omb2, gr), gr));
      least = fminf(least, v[c]);
      most = fmaxf(most, v[c]);
    }
    if (__any(least < 7.888609052210118e-31f || most == INFINITY)) {  // 2^-100; g^2 may overflow
#pragma unroll
      for (int c = 0; c < 8; ++c) r[c] = sqrtf(v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) r[c] = root_of(v[c]);
    }
    // the quotient by the hardware's reciprocal: within two ulps of the update
#pragma unroll
    for (int c = 0; c < 8; ++c)
      w[c] = w[c] * sc.keep - sc.rate * (m[c] * __builtin_amdgcn_rcpf(fmaf(r[c], sc.root, h.eps)));
    if (t.master) store8<GAP>(t.master, false, i, two, w);
    store8<GAP>(t.param, t.flags & 1, i, two, w);
    if constexpr (BITS == 32) {
      store8<GAP>(t.m, false, i, two, m);
      store8<GAP>(t.v, false, i, two, v);
    } else {
      const uint32_t key = mix(key0 + 0x85A308D3u * uint32_t(uint64_t(i) >> 32));
      const int bm = block_byte(block_max(m)), bv = block_byte(block_max(r));
      // 2^-k from its exponent bits: bytes are at most 247, so these are normal numbers
      const float im = __uint_as_float(uint32_t(254 - bm) << 23), iv = __uint_as_float(uint32_t(254 - bv) << 23);
      // An r above 0 gets a code above 0: below 2^-9 that is 1, the code of 2^-9.  Infinities get
      // the largest code.  Asked for by the smallest and largest v: r iv < 2^-9 only if v iv iv is
      // below 2^-17.
      if (__any((least * iv) * iv < 7.62939453125e-06f || most == INFINITY)) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          m[c] = fminf(fmaxf(m[c] * im, -448.f), 448.f);
          r[c] = r[c] > 0.f ? fminf(fmaxf(r[c] * iv, 0.001953125f), 448.f) : 0.f;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) m[c] *= im, r[c] *= iv;
      }
      uint32_t u[8], near = ~0u;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        u[c] = mix(uint32_t(i) + key + c);
        near = min(near, min(past(m[c], word_m(u[c]) + 0x2000u), past(r[c], word_v(u[c]) + 0x2000u)));
      }
      // One element of 2^18 lies so near a border that its roundings to fp32 would decide which
      // code it gets: there the state is taken in fp64.
      if (__any(near <= 0x3000u)) {
        uint32_t left = 0;  // bit c: m[c], bit 8 + c: r[c]
#pragma unroll
        for (int c = 0; c < 8; ++c)
          left |= uint32_t(at_border(m[c], word_m(u[c]))) << c | uint32_t(at_border(r[c], word_v(u[c]))) << (8 + c);
        while (left) {
          const int at = __builtin_ctz(left), root = at >> 3;
          const int64_t e = i + (at & 7);
          left &= left - 1;
          float y = 0.f;
          uint32_t word = 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (at == c) y = m[c], word = word_m(u[c]);
            if (at == 8 + c) y = r[c], word = word_v(u[c]);
          }
          // gradient and state anew from memory, so that neither is kept for this in registers
          const double g64 = double(t.flags & 2 ? bf2f(static_cast<const bf16_t*>(t.grad)[e]) : static_cast<const float*>(t.grad)[e]) * gs;
          const double s64 = ldexp(double(__builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(root ? t.v : t.m)[e], 0)),
                                   (root ? t.vs : t.ms)[e >> 7] - 127);
          const float border = __uint_as_float(__float_as_uint(fabsf(y)) - uint32_t(int(past(y, word)) >> 12));
          const double b = root ? h.beta2 : h.beta1;
          const double now = root ? (b * (s64 * s64) + (1. - b) * g64 * g64) * iv * iv : fabs(b * s64 + (1. - b) * g64) * im;
          const bool up = now >= (root ? double(border) * border : double(border));
          y = copysignf(up ? border : __uint_as_float(__float_as_uint(border) - 1u), y);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (at == c) m[c] = y;
            if (at == 8 + c) r[c] = y;
          }
        }
      }
      encode(m, r, u, cm, cv);
      store_codes(t.m, i, cnt, cm);
      store_codes(t.v, i, cnt, cv);
      if ((threadIdx.x & 15) == 0 && cnt) {
        t.ms[i >> 7] = uint8_t(bm);
        t.vs[i >> 7] = uint8_t(bv);
      }
    }
  };
  // FULL: the strip lies inside the tensor, so no element's place is asked for
  auto strip = [&](int64_t at, auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int64_t i = at + mine;
    auto left = [&](int64_t e) { return FULL || t.n - e >= 4 ? 4 : t.n > e ? int(t.n - e) : 0; };
    const int two[2] = {left(i), left(i + GAP)};
    const int cnt = two[0] + two[1];
    float g[8], w[8], m[8], v[8];
    load8<GAP>(t.grad, t.flags & 2, i, two, g);
    if (t.master) load8<GAP>(t.master, false, i, two, w);
    else load8<GAP>(t.param, t.flags & 1, i, two, w);
    if constexpr (BITS == 32) {
      load8<GAP>(t.m, false, i, two, m);
      load8<GAP>(t.v, false, i, two, v);
      update(i, two, g, w, m, v, uint2{}, uint2{}, 0.f, 0.f);
    } else {
      const uint2 cm = load_codes(t.m, i, cnt), cv = load_codes(t.v, i, cnt);
      const float sm = cnt ? pow2(int(t.ms[i >> 7]) - 127) : 0.f, sv = cnt ? pow2(int(t.vs[i >> 7]) - 127) : 0.f;
      update(i, two, g, w, m, v, cm, cv, sm, sv);
    }
  };
  const int64_t at = strip0 * kStrip;
  if (at + kStrip > t.n) {
    if (at < t.n) strip(at, std::false_type{});
  } else if constexpr (BITS == 32) {
    strip(at, std::true_type{});
  } else {
    // GB, WB: gradients, weights in bf16
    auto run = [&](auto gb, auto wb) {
      constexpr bool GB = decltype(gb)::value, WB = decltype(wb)::value;
      const char* gp = static_cast<const char*>(t.grad);
      const char* wp = t.master ? reinterpret_cast<const char*>(t.master) : static_cast<const char*>(t.param);
      auto load = [](const char* p, auto bf, float (&o)[8]) {
        if constexpr (decltype(bf)::value) {
          const uint4 q = *reinterpret_cast<const uint4*>(p);
          const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) o[2 * c] = __uint_as_float(u[c] << 16), o[2 * c + 1] = __uint_as_float(u[c] & 0xFFFF0000u);
        } else {
          const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 16);
          o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
        }
      };
      const int64_t i = at + mine;
      const int two[2] = {4, 4};
      float g[8], w[8], m[8], v[8];
      load(gp + i * (GB ? 2 : 4), gb, g);
      load(wp + i * (WB ? 2 : 4), wb, w);
      const uint2 cm = load_codes(t.m, i, 8), cv = load_codes(t.v, i, 8);
      update(i, two, g, w, m, v, cm, cv, pow2(int(t.ms[i >> 7]) - 127), pow2(int(t.vs[i >> 7]) - 127));
    };
    const bool wb = !t.master && (t.flags & 1);
    if (t.flags & 2) wb ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
    else wb ? run(std::false_type{}, std::true_type{}) : run(std::false_type{}, std::false_type{});
  }
}

hipError_t launch_adamw(const lc_moe_adamw_tensor* tensors, int count, const lc_moe_adamw_hyper& h, hipStream_t st) {
  using namespace aw;
  Args a{};
  a.h.lr = h.lr;
  a.h.beta1 = h.beta1;
  a.h.omb1 = static_cast<float>(1. - double(h.beta1));
  a.h.beta2 = h.beta2;
  a.h.omb2 = static_cast<float>(1. - double(h.beta2));
  a.h.eps = h.eps;
  a.h.seed = h.seed;
  a.h.step = h.step;
  a.h.step_dev = h.step_dev;
  a.h.grad_scale = h.grad_scale;
  a.h.p1 = power(double(h.beta1), h.step_dev ? 1 : h.step);
  a.h.p2 = power(double(h.beta2), h.step_dev ? 1 : h.step);
  // One launch covers up to kMaxTensors pieces and kMaxBlocks workgroups (the grid holds
  // 2^32 - 1 work-items); a tensor that needs more is cut between strips.
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
    const int64_t strips = (t.n + kStrip - 1) / kStrip;
    for (int64_t at = 0; at < strips;) {
      if (a.count == kMaxTensors || blocks == kMaxBlocks) {
        const hipError_t err = flush();
        if (err != hipSuccess) return err;
      }
      int64_t take = strips - at;
      if (take > kMaxBlocks - blocks) take = kMaxBlocks - blocks;
      a.first[a.count] = uint32_t(blocks);
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
      d.at = uint32_t(at);
      d.flags = (t.param_dtype == LC_MOE_BF16 ? 1u : 0u) | (t.grad_dtype == LC_MOE_BF16 ? 2u : 0u) | (uint32_t(i) << 2);
      blocks += take;
      at += take;
    }
  }
  return flush();
}

}  // namespace lcm
