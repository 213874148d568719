// Choice of experts from the router's logits, and the gradient of its gates
// (include/lc_moe_block.h): softmax or sigmoid scores, a bias for the choice, groups of experts,
// top-K, renormalised gates.
#include "block.h"
#include "topk.h"

namespace lcm {

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

struct SelectArgs {
  const float* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* gate;
  int T, E, K, score, groups, size, top_groups, rank, renorm;
  float scale;
};

// Gates of the picks, pick k in lane k (valid: there is one): x its logit.  m and sum: the
// softmax's largest logit and sum over the pool (not read with renorm or sigmoid scores).
__device__ __forceinline__ float pick_gate(const SelectArgs& a, bool valid, float x, float m, float sum) {
  if (a.renorm) {
    // shares of the picks from the logarithms of their scores, so that none underflows
    const float ls = a.score == LC_MOE_SOFTMAX ? x : fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
    const float top = __ockl_wfred_max_f32(valid ? ls : -INFINITY);
    const float w = valid ? expf(ls - top) : 0.f;
    return a.scale * (w / __ockl_wfred_add_f32(w));
  }
  const float s = a.score == LC_MOE_SOFTMAX ? expf(x - m) / sum : 1.f / (1.f + expf(-x));
  return a.scale * s;
}

// One token by one wavefront, scores in fp64.  c: room for E values in LDS.
__device__ void select_token_f64(const SelectArgs& a, int t, int lane, double* c) {
  const float* row = a.logits + size_t(t) * a.E;
  double m = -INFINITY, sum = 0.0;
  if (a.score == LC_MOE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 64) m = fmax(m, double(row[e]));
    m = wave_max(m);
    for (int e = lane; e < a.E; e += 64) sum += row[e] > -INFINITY ? exp(row[e] - m) : 0.0;
    sum = wave_sum(sum);
  }
  for (int e = lane; e < a.E; e += 64) {
    const float x = row[e], b = a.bias ? a.bias[e] : 0.f;
    const bool on = x > -INFINITY && b > -INFINITY;
    const double s = a.score == LC_MOE_SOFTMAX ? exp(x - m) / sum : 1.0 / (1.0 + exp(-double(x)));
    c[e] = on ? s + b : -INFINITY;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (a.top_groups < a.groups) {
    double best = -INFINITY;
    if (lane < a.groups) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int e = lane * a.size; e < (lane + 1) * a.size; ++e) {
        const double v = c[e];
        m2 = v > m1 ? m1 : v > m2 ? v : m2;
        m1 = v > m1 ? v : m1;
      }
      best = a.rank == 2 && m2 > -INFINITY ? m1 + m2 : m1;
    }
    unsigned long long kept = 0;
    for (int k = 0; k < a.top_groups; ++k) {
      const bool left = lane < a.groups && !(kept >> lane & 1);
      const double top = wave_max(left ? best : -INFINITY);
      const unsigned long long at = __ballot(left && best == top);
      kept |= at & (~at + 1);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int e = lane; e < a.E; e += 64)
      if (!(kept >> (e / a.size) & 1)) c[e] = -INFINITY;
  }
  int pick = -1;
  for (int k = 0; k < a.K; ++k) {
    double bv = -INFINITY;
    int be = 0x7fffffff;
    for (int e = lane; e < a.E; e += 64) {
      const bool better = c[e] > bv;
      bv = better ? c[e] : bv;
      be = better ? e : be;
    }
    const double top = wave_max(bv);
    const int e = __ockl_wfred_min_i32(bv == top ? be : 0x7fffffff);
    if (e == 0x7fffffff) break;  // nothing is left
    if (e % 64 == lane) c[e] = -INFINITY;
    pick = lane == k ? e : pick;
  }
  const float x = pick >= 0 ? row[pick] : 0.f;
  float g;
  if (a.renorm || a.score == LC_MOE_SIGMOID)
    g = pick_gate(a, pick >= 0, x, 0.f, 1.f);
  else
    g = float(double(a.scale) * (exp(x - m) / sum));
  if (lane < a.K) {
    a.idx[size_t(t) * a.K + lane] = pick;
    a.gate[size_t(t) * a.K + lane] = pick >= 0 ? g : 0.f;
  }
}

__global__ __launch_bounds__(64) void select_kernel(SelectArgs a) {
  extern __shared__ double c[];
  const int t = blockIdx.x, lane = threadIdx.x;
  if (a.mask && !a.mask[t]) {
    if (lane < a.K) {
      a.idx[size_t(t) * a.K + lane] = -1;
      a.gate[size_t(t) * a.K + lane] = 0.f;
    }
    return;
  }
  select_token_f64(a, t, lane, c);
}

hipError_t launch_select(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits, const float* bias,
                         const uint8_t* mask, int32_t* idx, float* gate, hipStream_t st) {
  const int E = s.N + s.Z;
  const SelectArgs a{logits, bias, mask, idx, gate, s.T, E, s.K, g.score, g.groups, E / g.groups, g.top_groups,
                     g.group_rank, g.renorm != 0, g.scale};
  select_kernel<<<dim3(s.T), dim3(64), size_t(E) * 8, st>>>(a);
  return hipGetLastError();
}

// ---- gradient ----------------------------------------------------------------------------

// One token by one wavefront; pick k in lane k.
__global__ __launch_bounds__(64) void select_backward_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ idx,
                                                             const float* __restrict__ dgate, const float* aux,
                                                             float* dlogits, int T, int E, int K, int score,
                                                             int renorm, float scale) {
  extern __shared__ float dp[];
  const int t = blockIdx.x, lane = threadIdx.x;
  const float* row = logits + size_t(t) * E;
  const int e = lane < K ? idx[size_t(t) * K + lane] : -1;
  const bool ok = static_cast<unsigned>(e) < static_cast<unsigned>(E);
  const float dg = ok ? dgate[size_t(t) * K + lane] : 0.f;
  const float x = ok ? row[e] : 0.f;
  const bool whole = score == LC_MOE_SOFTMAX && !renorm;
  float v;  // pick's own term
  if (renorm) {
    const float ls = score == LC_MOE_SOFTMAX ? x : fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
    const bool on = ok && ls > -INFINITY;
    const float top = __ockl_wfred_max_f32(on ? ls : -INFINITY);
    const float u = on ? expf(ls - top) : 0.f;
    const float sum = __ockl_wfred_add_f32(u);
    const float w = sum > 0.f ? u / sum : 0.f;
    const float mean = __ockl_wfred_add_f32(w * dg);
    v = scale * (w * (dg - mean));
    if (score == LC_MOE_SIGMOID) v *= 1.f / (1.f + expf(x));
  } else if (score == LC_MOE_SIGMOID) {
    const float s = 1.f / (1.f + expf(-x)), r = 1.f / (1.f + expf(x));
    v = scale * dg * (s * r);
  } else {
    v = scale * dg;
  }
  for (int i = lane; i < E; i += 64) dp[i] = 0.f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int k = 0; k < K; ++k)  // in pick order: an index may repeat
    if (lane == k && ok) dp[e] += v;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float m = -INFINITY, sum = 0.f, mean = 0.f;
  if (whole) {
    for (int i = lane; i < E; i += 64) m = fmaxf(m, row[i]);
    m = __ockl_wfred_max_f32(m);
    m = m > -INFINITY ? m : 0.f;
    for (int i = lane; i < E; i += 64) sum += expf(row[i] - m);
    sum = __ockl_wfred_add_f32(sum);
    const float p = sum > 0.f ? expf(x - m) / sum : 0.f;
    mean = __ockl_wfred_add_f32(ok ? p * v : 0.f);
  }
  for (int i = lane; i < E; i += 64) {
    float d = dp[i];
    if (whole) d = sum > 0.f ? expf(row[i] - m) / sum * (d - mean) : 0.f;
    if (aux) d += aux[size_t(t) * E + i];
    dlogits[size_t(t) * E + i] = d;
  }
}

hipError_t launch_select_backward(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits,
                                  const int32_t* idx, const float* dgate, const float* aux, float* dlogits,
                                  hipStream_t st) {
  const int E = s.N + s.Z;
  select_backward_kernel<<<dim3(s.T), dim3(64), size_t(E) * 4, st>>>(logits, idx, dgate, aux, dlogits, s.T, E, s.K,
                                                                     g.score, g.renorm != 0, g.scale);
  return hipGetLastError();
}

}  // namespace lcm
