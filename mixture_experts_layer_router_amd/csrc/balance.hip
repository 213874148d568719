// Load-balance loss, per-expert counts, z loss and their gradient with respect to the router
// logits (formulas in include/lc_moe_train.h).  No atomics on floating-point values: every sum
// has a fixed order.
//
// Three launches: softmax statistics of every token with each block's sums of probabilities
// and counts (the logits are read once); the sums over a sequence's blocks; the losses and the
// gradient (the logits are read again, from the memory-side cache where they fit).  With few
// blocks the last launch adds them itself, and few logits take one workgroup and one launch:
// there a launch's 5 us count.
//
// Bound by memory: T = 16384, E = 768, 8 sequences (50 MB of logits read twice, 50 MB of gradient
// written) takes 35.3 us: 16.5 for the statistics, 4 for the sums, 17 for the gradient (5.9 TB/s).  The
// statistics run at 3 TB/s: their arithmetic, about 17 operations a logit, takes 7 us, and 512
// blocks begin and end together; four rows of a wave loaded at once made it 37.8.  T = 64 takes
// 12.5 us of kernels, T = 4096 with E = 96 16, less than the two or three calls' own time.  Steps
// of the last form: the sequence found by one look at 64 bounds and u kept from token to token
// (38.4 -> 36.9), no question for -infinity beside the exponential's own (35.3).
#include "train.h"
#include "logit_row.h"

namespace lcm {

__device__ __forceinline__ int seq_bound(const int32_t* __restrict__ off, int i, int T) {
  if (!off) return i == 0 ? 0 : T;
  const int v = off[i];
  return v < 0 ? 0 : v > T ? T : v;
}

// 64 of the sequences' bounds in the lanes of a wave, so that finding a token's sequence and the
// ones behind it waits for memory once: lane l has bound base + l.
struct Bounds {
  int base, held;
  __device__ __forceinline__ void hold(const int32_t* __restrict__ off, int i, int S, int T, int lane) {
    base = i;
    held = seq_bound(off, i + lane < S ? i + lane : S, T);
  }
  __device__ __forceinline__ int at(const int32_t* __restrict__ off, int i, int T) const {
    const int l = __builtin_amdgcn_readfirstlane(i - base);
    return unsigned(l) < 64u ? __builtin_amdgcn_readlane(held, l) : seq_bound(off, i, T);
  }
};

struct BalArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* off;
  const uint8_t* mask;
  int S, T, E, K, n_eb;
  int tok, grad_tok;  // tokens of a workgroup: statistics, gradient
  float balance, z;
  TokStat* stat;
  float* part_p;
  int32_t* part_c;
  int32_t* part_n;
  float* part_z;
  int32_t* seq_n;
  float* seq_z;
  float* seq_loss;
  float* loss;
  int32_t* load;
  float* prob;
  float* dlogits;
};

// f[s][i] for c picks among n tokens: E c / (K n), in fp64 (whole numbers up to 2^36).
__device__ __forceinline__ float rel_load(int E, int K, int c, int n) {
  return static_cast<float>(double(E) * c / (double(K) * n));
}

// The losses from the sequences' numbers (one workgroup of THREADS; fixed order).
template <int THREADS>
__device__ __forceinline__ void write_losses(const BalArgs& a) {
  __shared__ double sl[THREADS], sz[THREADS];
  __shared__ long long sn[THREADS];
  __shared__ int sv[THREADS];
  double l = 0., z = 0.;
  long long n = 0;
  int live = 0;
  const int i = threadIdx.x;
  for (int s = i; s < a.S; s += THREADS) {
    n += a.seq_n[s];
    live += a.seq_n[s] > 0;
    z += a.seq_z[s];
    for (int b = 0; b < a.n_eb; ++b) l += a.seq_loss[size_t(s) * a.n_eb + b];
  }
  sl[i] = l, sz[i] = z, sn[i] = n, sv[i] = live;
  __syncthreads();
  for (int h = THREADS / 2; h > 0; h >>= 1) {
    if (i < h) sl[i] += sl[i + h], sz[i] += sz[i + h], sn[i] += sn[i + h], sv[i] += sv[i + h];
    __syncthreads();
  }
  if (i == 0) {
    a.loss[0] = sv[0] > 0 ? static_cast<float>(double(a.balance) / sv[0] * sl[0]) : 0.f;
    a.loss[1] = sn[0] > 0 && a.z != 0.f ? static_cast<float>(double(a.z) / double(sn[0]) * sz[0]) : 0.f;
  }
}

// The blocks of sequence s: b0 .. b1-1.
__device__ __forceinline__ void seq_blocks(const BalArgs& a, int s, int& b0, int& b1) {
  const int lo = seq_bound(a.off, s, a.T), up = seq_bound(a.off, s + 1, a.T);
  b0 = lo / a.tok;
  b1 = up > lo ? (up - 1) / a.tok + 1 : b0;
}

// u of sequence `seq` (its tokens that count: n > 0) in a wave's lanes.  live: sequences with such
// tokens.  ADD: the counts are added from the blocks'.
template <int EPL, int V, bool ADD>
__device__ __forceinline__ void load_u(const BalArgs& a, int seq, int n, int live, int lane, float (&u)[EPL]) {
  const long long kn = static_cast<long long>(a.K) * n;
  const float scale = a.balance / (static_cast<float>(live) * static_cast<float>(kn) * static_cast<float>(n));
  int b0 = 0, b1 = 1;
  if (ADD) seq_blocks(a, seq, b0, b1);
  const int32_t* cnt = ADD ? a.part_c + (size_t(b0) + seq) * a.E : a.load + size_t(seq) * a.E;
#pragma unroll
  for (int j = 0; j < EPL / V; ++j) {
    const int e = (j * 64 + lane) * V;
    int c[V] = {};
    if (e < a.E) {
#pragma unroll 8
      for (int b = 0; b < b1 - b0; ++b) {
        if constexpr (V == 4) {
          const int4 q = *reinterpret_cast<const int4*>(cnt + size_t(b) * a.E + e);
          c[0] += q.x, c[1] += q.y, c[2] += q.z, c[3] += q.w;
        } else {
          c[0] += cnt[size_t(b) * a.E + e];
        }
      }
    }
#pragma unroll
    for (int w = 0; w < V; ++w)
      u[j * V + w] = static_cast<float>(static_cast<long long>(a.E) * c[w] - kn) * scale;
  }
}

// Gradient of token t by one wave, p its logits.  total: all tokens that count.
template <int EPL, int V>
__device__ __forceinline__ void token_grad(const BalArgs& a, int t, int lane, float (&p)[EPL], const float (&u)[EPL],
                                           const TokStat& ts, float total) {
  float* out = a.dlogits + size_t(t) * a.E;
  if (ts.seq < 0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = 0.f;
    store_row<EPL, V>(out, a.E, lane, p);
    return;
  }
  const float zl = a.z != 0.f ? 2.f * a.z / total * ts.lse : 0.f;
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    p[i] = exp_neg(p[i] - ts.m) * ts.rs;
    dot += p[i] * u[i];
  }
  dot = __ockl_wfred_add_f32(dot);
#pragma unroll
  for (int i = 0; i < EPL; ++i) p[i] *= u[i] - dot + zl;
  store_row<EPL, V>(out, a.E, lane, p);
}

// One workgroup of up to WAVES waves per a.tok tokens, a wave per token.  ONE: the only
// workgroup; it finishes the sums, the losses and the gradient as well.
template <int EPL, int V, int WAVES, bool ONE>
__global__ __launch_bounds__(WAVES * 64) void balance_tokens_kernel(BalArgs a) {
  __shared__ __attribute__((aligned(16))) float ps[WAVES][EPL * 64];  // a wave's sums of p
  __shared__ int32_t cnt[EPL * 64];
  __shared__ int wn[WAVES];
  __shared__ float wz[WAVES], wl[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = a.T, E = a.E, K = a.K;
  const int waves = blockDim.x >> 6, threads = blockDim.x;
  const int t0 = blockIdx.x * a.tok, t1 = t0 + a.tok < T ? t0 + a.tok : T;
  // bit l: token t0 + l is not masked (a workgroup has at most 64)
  const unsigned long long marked = __ballot(t0 + lane < t1 && (!a.mask || a.mask[t0 + lane]));
  int s = 0;
  Bounds bounds;
  if (!ONE) {  // the first sequence that ends behind t0 (S: none), 64 ends at a time
    int last = a.S;
    while (last - s > 62) {
      const int step = (last - s + 63) >> 6, e = s + (lane + 1) * step;
      const unsigned long long b = __ballot(seq_bound(a.off, e < last ? e : last, T) > t0);
      if (!b) {
        s = last;
        break;
      }
      s += __builtin_ctzll(b) * step;
      last = s + step - 1 < last ? s + step - 1 : last;
    }
    bounds.hold(a.off, s, a.S, T, lane);
    const unsigned long long b = __ballot(lane > 0 && s + lane <= a.S && bounds.held > t0);
    s = b ? s + __builtin_ctzll(b) - 1 : a.S;
  } else {
    bounds.hold(a.off, 0, a.S, T, lane);
  }
  int done = t0;  // tokens before this one are dealt with
  for (; s < a.S; ++s) {
    const int lo = bounds.at(a.off, s, T), up = bounds.at(a.off, s + 1, T);
    if (!ONE && lo >= t1) break;
    const int first = lo > done ? lo : done, b = up < t1 ? up : t1;
    const int tokens = b > first ? b - first : 0;
    if (!ONE && tokens == 0) continue;
    for (int t = done + tid; t < first && tokens; t += threads) a.stat[t] = TokStat{0.f, 0.f, 0.f, -1};
    if (tokens) done = b;
    for (int e = tid; e < E; e += threads) cnt[e] = 0;
    __syncthreads();
    float acc[EPL], v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    int n = 0;
    float z = 0.f;
    // the next token's row and picks are on their way while this one's are worked on
    float nxt[EPL];
    bool take = false;
    int t = first + wave, npick = -1;
    auto fetch = [&](int at) {
      take = marked >> (at - t0) & 1;
      if (!take) return;
      load_row<EPL, V>(a.logits + size_t(at) * E, E, lane, -INFINITY, nxt);
      if (lane < K) npick = a.idx[size_t(at) * K + lane];
    };
    if (t < b) fetch(t);
    for (; t < b; t += waves) {
      const bool now = take;
      const int pick = lane < K ? npick : -1;
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = nxt[i];
      if (t + waves < b) fetch(t + waves);
      TokStat ts{0.f, 0.f, 0.f, -1};
      if (now) {
        const RowSum r = softmax_row<EPL>(v);
        if (r.m > -INFINITY) {
          const float rs = 1.f / r.sum, lse = r.m + logf(r.sum);
#pragma unroll
          for (int i = 0; i < EPL; ++i) acc[i] = fmaf(v[i], rs, acc[i]);
          n += 1;
          z += lse * lse;
          ts = TokStat{r.m, rs, lse, s};
          if (unsigned(pick) < unsigned(E)) atomicAdd(&cnt[pick], 1);
          for (int k = lane + 64; k < K; k += 64) {
            const int e = a.idx[size_t(t) * K + k];
            if (unsigned(e) < unsigned(E)) atomicAdd(&cnt[e], 1);
          }
        }
      }
      if (lane == 0) a.stat[t] = ts;
    }
    const int used = tokens < waves ? tokens : waves;  // waves that had a token
    if (wave < used) store_row<EPL, V>(ps[wave], E, lane, acc);
    if (lane == 0) wn[wave] = n, wz[wave] = z;
    __syncthreads();
    int nsum = 0;
    float zsum = 0.f;
    for (int w = 0; w < used; ++w) nsum += wn[w], zsum += wz[w];
    if constexpr (ONE) {
      float term = 0.f;
      for (int e = tid; e < E; e += threads) {
        float p = 0.f;
        for (int w = 0; w < used; ++w) p += ps[w][e];
        const float mean = nsum > 0 ? p / static_cast<float>(nsum) : 0.f;
        a.load[size_t(s) * E + e] = cnt[e];
        a.prob[size_t(s) * E + e] = mean;
        if (nsum > 0) term += rel_load(E, K, cnt[e], nsum) * mean;
      }
      term = __ockl_wfred_add_f32(term);
      if (lane == 0) wl[wave] = term;
      __syncthreads();
      if (tid == 0) {
        float l = 0.f;
        for (int w = 0; w < waves; ++w) l += wl[w];
        a.seq_loss[s] = l;
        a.seq_n[s] = nsum;
        a.seq_z[s] = zsum;
      }
    } else {
      const size_t row = size_t(blockIdx.x) + s;
      for (int e = tid; e < E; e += threads) {
        float p = 0.f;
        for (int w = 0; w < used; ++w) p += ps[w][e];
        a.part_p[row * E + e] = p;
        a.part_c[row * E + e] = cnt[e];
      }
      if (tid == 0) {
        a.part_n[row] = nsum;
        a.part_z[row] = zsum;
      }
    }
    __syncthreads();
  }
  for (int t = done + tid; t < t1; t += threads) a.stat[t] = TokStat{0.f, 0.f, 0.f, -1};
  if constexpr (ONE) {
    __threadfence_block();
    __syncthreads();
    if (a.dlogits) {
      long long total = 0;
      int live = 0;
      for (int q = 0; q < a.S; ++q) {
        const int n = a.seq_n[q];
        total += n;
        live += n > 0;
      }
      int have = -1;  // the sequence that u belongs to
      float u[EPL];
      for (int t = wave; t < T; t += waves) {
        const TokStat ts = a.stat[t];
        float v[EPL];
        if (ts.seq >= 0) load_row<EPL, V>(a.logits + size_t(t) * E, E, lane, -INFINITY, v);
        if (ts.seq >= 0 && ts.seq != have) load_u<EPL, V, false>(a, have = ts.seq, a.seq_n[ts.seq], live, lane, u);
        token_grad<EPL, V>(a, t, lane, v, u, ts, static_cast<float>(total));
      }
    }
    write_losses<WAVES * 64>(a);
  }
}

// Sums over a sequence's blocks: workgroup (64 experts, sequence); the 16 waves take every
// sixteenth block each and are added in wave order.
__global__ __launch_bounds__(1024) void balance_sums_kernel(BalArgs a) {
  __shared__ float sp[16][64], sz[16];
  __shared__ int sc[16][64], sn[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.y, e = blockIdx.x * 64 + lane, E = a.E;
  int b0, b1;
  seq_blocks(a, s, b0, b1);
  const int ec = e < E ? e : E - 1;  // lanes past E repeat the last expert; never written
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
#pragma unroll 4
  for (int b = b0 + wave; b < b1; b += 16) {
    const size_t row = size_t(b) + s;
    p += a.part_p[row * E + ec];
    c += a.part_c[row * E + ec];
    n += a.part_n[row];
    z += a.part_z[row];
  }
  sp[wave][lane] = p;
  sc[wave][lane] = c;
  if (lane == 0) sn[wave] = n, sz[wave] = z;
  __syncthreads();
  if (wave != 0) return;
  p = z = 0.f;
  c = n = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) p += sp[w][lane], c += sc[w][lane], n += sn[w], z += sz[w];
  float term = 0.f;
  if (e < E) {
    const float mean = n > 0 ? p / static_cast<float>(n) : 0.f;
    a.load[size_t(s) * E + e] = c;
    a.prob[size_t(s) * E + e] = mean;
    if (n > 0) term = rel_load(E, a.K, c, n) * mean;
  }
  term = __ockl_wfred_add_f32(term);
  if (lane == 0) {
    a.seq_loss[size_t(s) * a.n_eb + blockIdx.x] = term;
    if (blockIdx.x == 0) {
      a.seq_n[s] = n;
      a.seq_z[s] = z;
    }
  }
}

// Few blocks and sequences (they are taken one after another): the sums in the last launch.
constexpr int kFewBlocks = 32, kFewSeqs = 2;

// Workgroup 0 of the last launch with few blocks: load, prob and the losses.
__device__ __forceinline__ void few_sums(const BalArgs& a) {
  __shared__ double sl[256], sz[256];
  __shared__ int sn[256], sv[256];
  const int i = threadIdx.x, E = a.E;
  double l = 0., z = 0.;
  int total = 0, live = 0;
  for (int s = 0; s < a.S; ++s) {
    int b0, b1, n = 0;
    seq_blocks(a, s, b0, b1);
    float zs = 0.f;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) n += a.part_n[b + s], zs += a.part_z[b + s];
    if (i == 0) {
      z += zs;
      total += n;
      live += n > 0;
    }
    for (int e = i; e < E; e += 256) {
      float p = 0.f;
      int c = 0;
#pragma unroll 8
      for (int b = b0; b < b1; ++b) {
        p += a.part_p[(size_t(b) + s) * E + e];
        c += a.part_c[(size_t(b) + s) * E + e];
      }
      const float mean = n > 0 ? p / static_cast<float>(n) : 0.f;
      a.load[size_t(s) * E + e] = c;
      a.prob[size_t(s) * E + e] = mean;
      if (n > 0) l += rel_load(E, a.K, c, n) * mean;
    }
  }
  sl[i] = l, sz[i] = z, sn[i] = total, sv[i] = live;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if (i < h) sl[i] += sl[i + h], sz[i] += sz[i + h], sn[i] += sn[i + h], sv[i] += sv[i + h];
    __syncthreads();
  }
  if (i == 0) {
    a.loss[0] = sv[0] > 0 ? static_cast<float>(double(a.balance) / sv[0] * sl[0]) : 0.f;
    a.loss[1] = sn[0] > 0 && a.z != 0.f ? static_cast<float>(double(a.z) / double(sn[0]) * sz[0]) : 0.f;
  }
}

// Workgroup 0: the losses.  The others: the gradient.  FEW: see above.
template <int EPL, int V, bool FEW>
__global__ __launch_bounds__(256) void balance_grad_kernel(BalArgs a) {
  if (blockIdx.x == 0) {
    if constexpr (FEW) few_sums(a);
    else write_losses<256>(a);
    return;
  }
  __shared__ int wt[4], wl[4], ns[FEW ? kFewSeqs : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int t = (int(blockIdx.x) - 1) * a.grad_tok + wave;
  const int t1 = int(blockIdx.x) * a.grad_tok < a.T ? int(blockIdx.x) * a.grad_tok : a.T;
  // the wave's tokens t, t + 4, ..: lane l has the statistics of the l-th
  TokStat held{0.f, 0.f, 0.f, -1};
  if (t + 4 * lane < t1) held = a.stat[t + 4 * lane];
  auto stat_of = [&](int l) {
    auto f = [&](float x) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l)); };
    return TokStat{f(held.m), f(held.rs), f(held.lse), __builtin_amdgcn_readlane(held.seq, l)};
  };
  float nxt[EPL], v[EPL], u[EPL];
  TokStat nts = stat_of(0);
  if (nts.seq >= 0) load_row<EPL, V>(a.logits + size_t(t) * a.E, a.E, lane, -INFINITY, nxt);
  int total = 0, live = 0;  // tokens that count: at most T
  for (int s = tid; s < a.S; s += 256) {
    int n = 0;
    if constexpr (FEW) {
      int b0, b1;
      seq_blocks(a, s, b0, b1);
#pragma unroll 8
      for (int b = b0; b < b1; ++b) n += a.part_n[b + s];
      ns[s] = n;
    } else {
      n = a.seq_n[s];
    }
    total += n;
    live += n > 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o), live += __shfl_xor(live, o);
  if (lane == 0) wt[wave] = total, wl[wave] = live;
  __syncthreads();
  total = wt[0] + wt[1] + wt[2] + wt[3];
  live = wl[0] + wl[1] + wl[2] + wl[3];
  int have = -1;  // the sequence that u belongs to
  for (int l = 0; t < t1; t += 4) {
    const TokStat ts = nts;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = nxt[i];
    if (t + 4 < t1) {
      nts = stat_of(++l);
      if (nts.seq >= 0) load_row<EPL, V>(a.logits + size_t(t + 4) * a.E, a.E, lane, -INFINITY, nxt);
    }
    if (ts.seq >= 0 && ts.seq != have)
      load_u<EPL, V, FEW>(a, have = ts.seq, FEW ? ns[ts.seq] : a.seq_n[ts.seq], live, lane, u);
    token_grad<EPL, V>(a, t, lane, v, u, ts, static_cast<float>(total));
  }
}

template <int EPL, int V>
static void launch_passes(const BalArgs& a, const BalPlan& p, hipStream_t st) {
  // most waves of a workgroup: LDS holds one row of sums for each, at most 64 KB in all
  // (T = 16384, E = 768: 35.3 us with 8 waves and 32 tokens, 36.3 with 4 waves, 39 with 16)
  constexpr int WAVES = EPL <= 32 ? 8 : 4;
  if (p.one) {
    hipLaunchKernelGGL((balance_tokens_kernel<EPL, V, WAVES, true>), dim3(1), dim3(WAVES * 64), 0, st, a);
    return;
  }
  const int waves = p.tok < WAVES ? p.tok : WAVES;
  hipLaunchKernelGGL((balance_tokens_kernel<EPL, V, WAVES, false>), dim3(p.nblocks), dim3(waves * 64), 0, st, a);
  const dim3 grid(1 + (a.dlogits ? (a.T + a.grad_tok - 1) / a.grad_tok : 0));
  if (p.nblocks <= kFewBlocks && a.S <= kFewSeqs) {
    hipLaunchKernelGGL((balance_grad_kernel<EPL, V, true>), grid, dim3(256), 0, st, a);
    return;
  }
  hipLaunchKernelGGL(balance_sums_kernel, dim3(p.n_eb, a.S), dim3(1024), 0, st, a);
  hipLaunchKernelGGL((balance_grad_kernel<EPL, V, false>), grid, dim3(256), 0, st, a);
}

hipError_t launch_balance_loss(const lc_moe_shape& s, const BalPlan& p, void* ws, float balance, float z,
                               const float* logits, const int32_t* idx, const int32_t* offsets, int S,
                               const uint8_t* mask, float* loss, int32_t* load, float* prob, float* dlogits,
                               hipStream_t st) {
  const int E = s.N + s.Z, epl = (E + 63) / 64;
  char* w = static_cast<char*>(ws);
  BalArgs a{};
  a.logits = logits;
  a.idx = idx;
  a.off = offsets;
  a.mask = mask;
  a.S = S;
  a.T = s.T;
  a.E = E;
  a.K = s.K;
  a.n_eb = p.one ? 1 : p.n_eb;
  a.tok = p.tok;
  // enough workgroups to fill the chip, then four tokens a wave (T = 16384, E = 768: 35.3 us; two
  // 36.5, eight 36.9)
  a.grad_tok = s.T < 8192 ? 4 : 16;
  a.balance = balance;
  a.z = z;
  a.stat = reinterpret_cast<TokStat*>(w + p.stat);
  a.part_p = reinterpret_cast<float*>(w + p.part_p);
  a.part_c = reinterpret_cast<int32_t*>(w + p.part_c);
  a.part_n = reinterpret_cast<int32_t*>(w + p.part_n);
  a.part_z = reinterpret_cast<float*>(w + p.part_z);
  a.seq_n = reinterpret_cast<int32_t*>(w + p.seq_n);
  a.seq_z = reinterpret_cast<float*>(w + p.seq_z);
  a.seq_loss = reinterpret_cast<float*>(w + p.seq_loss);
  a.loss = loss;
  a.load = load;
  a.prob = prob;
  a.dlogits = dlogits;
  if (E % 4 == 0) {
    if (epl <= 4) launch_passes<4, 4>(a, p, st);
    else if (epl <= 8) launch_passes<8, 4>(a, p, st);
    else if (epl <= 12) launch_passes<12, 4>(a, p, st);
    else if (epl <= 16) launch_passes<16, 4>(a, p, st);
    else if (epl <= 32) launch_passes<32, 4>(a, p, st);
    else launch_passes<64, 4>(a, p, st);
  } else {
    if (epl <= 2) launch_passes<2, 1>(a, p, st);
    else if (epl <= 8) launch_passes<8, 1>(a, p, st);
    else if (epl <= 16) launch_passes<16, 1>(a, p, st);
    else if (epl <= 32) launch_passes<32, 1>(a, p, st);
    else launch_passes<64, 1>(a, p, st);
  }
  return hipGetLastError();
}

}  // namespace lcm
