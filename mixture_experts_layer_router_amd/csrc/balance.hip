// Load-balance loss, per-expert counts, z loss and their gradient with respect to the router
// logits (formulas in include/lc_moe_train.h).  Three passes: per-token softmax statistics
// and per-block sums of the probabilities and counts; the sums over a sequence's blocks;
// the gradient.  No atomics on floating-point values: every sum has a fixed order.
#include "train.h"
#include "topk.h"

namespace lcm {

__device__ __forceinline__ int seq_bound(const int32_t* __restrict__ off, int i, int T) {
  if (!off) return i == 0 ? 0 : T;
  const int v = off[i];
  return v < 0 ? 0 : v > T ? T : v;
}

// One workgroup per kBalTok tokens, one wave per token at a time; expert e in lane e % 64.
template <int EPL>
__global__ __launch_bounds__(256) void balance_tokens_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const int32_t* __restrict__ off, int S,
    const uint8_t* __restrict__ mask, int T, int E, int K, TokStat* __restrict__ stat, float* __restrict__ part_p,
    int32_t* __restrict__ part_c, int32_t* __restrict__ part_n, float* __restrict__ part_z) {
  extern __shared__ int32_t lds[];
  int32_t* cnt = lds;                                // [E]
  float* ps = reinterpret_cast<float*>(lds + E);     // [E]
  __shared__ int wn[4];
  __shared__ float wz[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * kBalTok, t1 = t0 + kBalTok < T ? t0 + kBalTok : T;
  // the first sequence that ends behind t0
  int s = 0, hi = S;
  while (s < hi) {
    const int mid = (s + hi) >> 1;
    if (seq_bound(off, mid + 1, T) > t0) hi = mid;
    else s = mid + 1;
  }
  int done = t0;  // tokens before this one are dealt with
  for (; s < S; ++s) {
    const int lo = seq_bound(off, s, T), up = seq_bound(off, s + 1, T);
    if (lo >= t1) break;
    const int a = lo > done ? lo : done, b = up < t1 ? up : t1;
    if (a >= b) continue;
    for (int t = done + tid; t < a; t += 256) stat[t] = TokStat{0.f, 0.f, 0.f, -1};
    done = b;
    for (int e = tid; e < E; e += 256) cnt[e] = 0;
    __syncthreads();
    float acc[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
    int n = 0;
    float z = 0.f;
    for (int t = a + wave; t < b; t += 4) {
      TokStat ts{0.f, 0.f, 0.f, -1};
      if (!mask || mask[t]) {
        float v[EPL], m = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int e = lane + 64 * j;
          v[j] = e < E ? logits[size_t(t) * E + e] : -INFINITY;
          m = fmaxf(m, v[j]);
        }
        m = __ockl_wfred_max_f32(m);
        if (m > -INFINITY) {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            v[j] = expf(v[j] - m);
            sum += v[j];
          }
          sum = __ockl_wfred_add_f32(sum);
          const float rs = 1.f / sum, lse = m + logf(sum);
#pragma unroll
          for (int j = 0; j < EPL; ++j) acc[j] += v[j] * rs;
          n += 1;
          z += lse * lse;
          ts = TokStat{m, rs, lse, s};
          for (int k = lane; k < K; k += 64) {
            const int e = idx[size_t(t) * K + k];
            if (unsigned(e) < unsigned(E)) atomicAdd(&cnt[e], 1);
          }
        }
      }
      if (lane == 0) stat[t] = ts;
    }
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int e = lane + 64 * j;
          if (e < E) ps[e] = w == 0 ? acc[j] : ps[e] + acc[j];
        }
      }
      __syncthreads();
    }
    if (lane == 0) {
      wn[wave] = n;
      wz[wave] = z;
    }
    __syncthreads();
    const size_t row = size_t(blockIdx.x) + s;
    for (int e = tid; e < E; e += 256) {
      part_p[row * E + e] = ps[e];
      part_c[row * E + e] = cnt[e];
    }
    if (tid == 0) {
      part_n[row] = wn[0] + wn[1] + wn[2] + wn[3];
      part_z[row] = (wz[0] + wz[1]) + (wz[2] + wz[3]);
    }
    __syncthreads();
  }
  for (int t = done + tid; t < t1; t += 256) stat[t] = TokStat{0.f, 0.f, 0.f, -1};
}

// Sums over a sequence's blocks: workgroup (block of 64 experts, sequence); wave w takes every
// fourth block, the four are added in wave order.
__global__ __launch_bounds__(256) void balance_sums_kernel(
    const int32_t* __restrict__ off, int T, int E, int K, const float* __restrict__ part_p,
    const int32_t* __restrict__ part_c, const int32_t* __restrict__ part_n, const float* __restrict__ part_z,
    int32_t* __restrict__ load, float* __restrict__ prob, int32_t* __restrict__ seq_n, float* __restrict__ seq_z,
    float* __restrict__ seq_loss) {
  __shared__ float sp[4][64];
  __shared__ int sc[4][64], sn[4];
  __shared__ float sz[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.y, e = blockIdx.x * 64 + lane;
  const int lo = seq_bound(off, s, T), up = seq_bound(off, s + 1, T);
  const int b0 = lo / kBalTok, b1 = up > lo ? (up - 1) / kBalTok + 1 : b0;
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
  for (int b = b0 + wave; b < b1; b += 4) {
    const size_t row = size_t(b) + s;
    if (e < E) {
      p += part_p[row * E + e];
      c += part_c[row * E + e];
    }
    n += part_n[row];
    z += part_z[row];
  }
  sp[wave][lane] = p;
  sc[wave][lane] = c;
  if (lane == 0) {
    sn[wave] = n;
    sz[wave] = z;
  }
  __syncthreads();
  if (wave != 0) return;
  n = sn[0] + sn[1] + sn[2] + sn[3];
  p = (sp[0][lane] + sp[1][lane]) + (sp[2][lane] + sp[3][lane]);
  c = sc[0][lane] + sc[1][lane] + sc[2][lane] + sc[3][lane];
  float term = 0.f;
  if (e < E) {
    const float mean = n > 0 ? p / static_cast<float>(n) : 0.f;
    load[size_t(s) * E + e] = c;
    prob[size_t(s) * E + e] = mean;
    if (n > 0) term = static_cast<float>(double(E) * c / (double(K) * n)) * mean;
  }
  term = __ockl_wfred_add_f32(term);
  if (lane == 0) {
    seq_loss[size_t(s) * gridDim.x + blockIdx.x] = term;
    if (blockIdx.x == 0) {
      seq_n[s] = n;
      seq_z[s] = (sz[0] + sz[1]) + (sz[2] + sz[3]);
    }
  }
}

// Totals over the sequences (one workgroup), the losses, and the gradient's two factors.
__global__ __launch_bounds__(256) void balance_loss_kernel(int S, int n_eb, float balance, float zc,
                                                           int32_t* __restrict__ seq_n,
                                                           const float* __restrict__ seq_z,
                                                           const float* __restrict__ seq_loss,
                                                           float* __restrict__ loss, float* __restrict__ factors) {
  __shared__ double sl[256], sz[256];
  __shared__ long long sn[256];
  __shared__ int sv[256];
  double l = 0., z = 0.;
  long long n = 0;
  int live = 0;
  for (int s = threadIdx.x; s < S; s += 256) {
    n += seq_n[s];
    live += seq_n[s] > 0;
    z += seq_z[s];
    for (int b = 0; b < n_eb; ++b) l += seq_loss[size_t(s) * n_eb + b];
  }
  const int i = threadIdx.x;
  sl[i] = l;
  sz[i] = z;
  sn[i] = n;
  sv[i] = live;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if (i < h) {
      sl[i] += sl[i + h];
      sz[i] += sz[i + h];
      sn[i] += sn[i + h];
      sv[i] += sv[i + h];
    }
    __syncthreads();
  }
  if (i == 0) {
    loss[0] = sv[0] > 0 ? static_cast<float>(double(balance) / sv[0] * sl[0]) : 0.f;
    loss[1] = sn[0] > 0 && zc != 0.f ? static_cast<float>(double(zc) / double(sn[0]) * sz[0]) : 0.f;
    factors[0] = sv[0] > 0 ? static_cast<float>(double(balance) / sv[0]) : 0.f;
    factors[1] = sn[0] > 0 ? static_cast<float>(2. * double(zc) / double(sn[0])) : 0.f;
  }
}

// dlogits: one wave per token.
template <int EPL>
__global__ __launch_bounds__(256) void balance_grad_kernel(const float* __restrict__ logits, int T, int E, int K,
                                                           const TokStat* __restrict__ stat,
                                                           const int32_t* __restrict__ load,
                                                           const int32_t* __restrict__ seq_n,
                                                           const float* __restrict__ factors,
                                                           float* __restrict__ dlogits) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (t >= T) return;
  const TokStat ts = stat[t];
  float* out = dlogits + size_t(t) * E;
  if (ts.seq < 0) {
    for (int e = lane; e < E; e += 64) out[e] = 0.f;
    return;
  }
  const int n = seq_n[ts.seq];
  const long long kn = static_cast<long long>(K) * n;
  const float scale = factors[0] / (static_cast<float>(kn) * static_cast<float>(n));
  const float zl = factors[1] != 0.f ? factors[1] * ts.lse : 0.f;
  float p[EPL], u[EPL], dot = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    p[j] = e < E ? expf(logits[size_t(t) * E + e] - ts.m) * ts.rs : 0.f;
    u[j] = e < E ? static_cast<float>(static_cast<long long>(E) * load[size_t(ts.seq) * E + e] - kn) * scale : 0.f;
    dot += p[j] * u[j];
  }
  dot = __ockl_wfred_add_f32(dot);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    if (e < E) out[e] = p[j] * (u[j] - dot + zl);
  }
}

hipError_t launch_balance_loss(const lc_moe_shape& s, const BalPlan& p, void* ws, float balance, float z,
                               const float* logits, const int32_t* idx, const int32_t* offsets, int S,
                               const uint8_t* mask, float* loss, int32_t* load, float* prob, float* dlogits,
                               hipStream_t st) {
  const int E = s.N + s.Z, epl = (E + 63) / 64;
  char* w = static_cast<char*>(ws);
  TokStat* stat = reinterpret_cast<TokStat*>(w + p.stat);
  float* part_p = reinterpret_cast<float*>(w + p.part_p);
  int32_t* part_c = reinterpret_cast<int32_t*>(w + p.part_c);
  int32_t* part_n = reinterpret_cast<int32_t*>(w + p.part_n);
  float* part_z = reinterpret_cast<float*>(w + p.part_z);
  int32_t* seq_n = reinterpret_cast<int32_t*>(w + p.seq_n);
  float* seq_z = reinterpret_cast<float*>(w + p.seq_z);
  float* seq_loss = reinterpret_cast<float*>(w + p.seq_loss);
  float* factors = reinterpret_cast<float*>(w + p.factors);
#define LCM_EPL(launch)            \
  if (epl <= 2) launch(2);         \
  else if (epl <= 4) launch(4);    \
  else if (epl <= 8) launch(8);    \
  else if (epl <= 16) launch(16);  \
  else if (epl <= 32) launch(32);  \
  else launch(64);
#define LCM_TOKENS(n)                                                                                       \
  hipLaunchKernelGGL(balance_tokens_kernel<n>, dim3(p.nblocks), dim3(256), size_t(E) * 8, st, logits, idx, \
                     offsets, S, mask, s.T, E, s.K, stat, part_p, part_c, part_n, part_z)
  LCM_EPL(LCM_TOKENS)
  hipLaunchKernelGGL(balance_sums_kernel, dim3(p.n_eb, S), dim3(256), 0, st, offsets, s.T, E, s.K, part_p, part_c,
                     part_n, part_z, load, prob, seq_n, seq_z, seq_loss);
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(256), 0, st, S, p.n_eb, balance, z, seq_n, seq_z, seq_loss,
                     loss, factors);
  if (dlogits) {
#define LCM_GRAD(n)                                                                                              \
  hipLaunchKernelGGL(balance_grad_kernel<n>, dim3((s.T + 3) / 4), dim3(256), 0, st, logits, s.T, E, s.K, stat, \
                     load, seq_n, factors, dlogits)
    LCM_EPL(LCM_GRAD)
  }
  return hipGetLastError();
}

}  // namespace lcm
