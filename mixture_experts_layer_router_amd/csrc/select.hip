// Choice of experts from the router's logits, and the gradient of its gates
// (include/lc_moe_block.h): softmax or sigmoid scores, a bias for the choice, groups of experts,
// top-K, renormalised gates.  One wavefront a token.
//
// Measured at T = 16384, E = 768: the choice (K = 12, sigmoid, 8 groups) takes 28-30 us by trace with the logits
// in the last-level cache, 32 a call then and 37-39 with other logits in every call; the vector units bound it:
// 820 instructions a token fill 53 of its 66 thousand cycles.  Softmax without groups 21 (call 22).  Where fp64
// decides for every token it takes 120 (all scores equal), and 297 with K = 64, where more than 64 scores are
// not below the bound (K above about 40).  The gradient takes 20-21 us (5 TB/s).
#include "block.h"
#include "logit_row.h"

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
    // Shares of the picks, a power of e taken out of their scores so that none underflows: a softmax
    // score is e^(x - top) of the largest, a sigmoid one e^min(x, 0) / (1 + e^-|x|).
    const bool soft = a.score == LC_MOE_SOFTMAX;
    const float l = soft ? x : fminf(x, 0.f);
    const float top = __ockl_wfred_max_f32(valid ? l : -INFINITY);
    float w = valid ? exp_neg(l - top) : 0.f;
    if (!soft) w *= 1.f / (1.f + exp_neg(-fabsf(x)));
    return w * (a.scale / __ockl_wfred_add_f32(w));
  }
  const float s = a.score == LC_MOE_SOFTMAX ? expf(x - m) / sum : 1.f / (1.f + expf(-x));
  return a.scale * s;
}

// Writes a token's places, pick k (-1: none) in lane k.
__device__ __forceinline__ void put_picks(const SelectArgs& a, int t, int lane, int pick, float g) {
  if (lane < a.K) {
    a.idx[size_t(t) * a.K + lane] = pick;
    a.gate[size_t(t) * a.K + lane] = pick >= 0 ? g : 0.f;
  }
}

// One token by one wavefront, scores in fp64.  c: room for E values in LDS.
__device__ __forceinline__ void select_token_f64(const SelectArgs& a, int t, int lane, double* c) {
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
  put_picks(a, t, lane, pick, g);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(u), lane), hi = __builtin_amdgcn_readlane(uint32_t(u >> 32), lane);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Sums of v over the lanes up to this one: within runs of 16 lanes, then the last lane of a run to the
// next run, and that of the lower half to the upper one.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // a lane's value to the next lane of its run
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // two on
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // four
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // eight
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lanes 15 and 47 to the runs behind them
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return v;
}

// Of the n values c of lanes 0 .. n-1 (n <= 64): how many are ahead of the lane's in descending order,
// equal ones in the order of their experts e.
__device__ __forceinline__ int place_of(double c, int e, int n) {
  int place = 0;
  for (int j = 0; j < n; ++j) {
    const double cj = lane_value(c, j);
    const int ej = __builtin_amdgcn_readlane(e, j);
    place += (cj > c || (cj == c && ej < e)) ? 1 : 0;
  }
  return place;
}
// The same in fp32 (-infinity in the lanes behind), but that equal ones get one place.
__device__ __forceinline__ int place_of(float c, int n) {
  int place = 0;
  for (int j = 0; j < n; j += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) place += lane_value(c, j + i) > c ? 1 : 0;
  }
  return place;
}

// Scores in fp32, a lane's EPL experts in registers (logit_row.h).  What may be picked is little:
// the K-th largest of the largest of 16 parts of the pool (64 for K above 16, and where 16 leave too
// many) bounds the K-th largest of all from below, and about 25 of 768 scores are not below it (K =
// 12); they are gathered one to a lane and sorted by counting.
// Where two scores next to each other are within the error of their fp32 values, the gathered ones
// are taken again in fp64; where two groups at the border are, or more than 64 scores are gathered
// (equal logits, say), the whole token is (select_token_f64).
template <int EPL, int V>
__global__ __launch_bounds__(256) void select_kernel(SelectArgs a, int room) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * (blockDim.x >> 6) + wave;
  if (t >= a.T) return;
  if (a.mask && !a.mask[t]) {
    put_picks(a, t, lane, -1, 0.f);
    return;
  }
  unsigned char* mine = lds + size_t(wave) * room;
  float x[EPL], c[EPL];
  load_row<EPL, V>(a.logits + size_t(t) * a.E, a.E, lane, -INFINITY, x);
  if (a.bias) {
    load_row<EPL, V>(a.bias, a.E, lane, 0.f, c);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = 0.f;
  }
  float m = -INFINITY;  // (of those that are numbers)
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = fmaxf(m, x[i]);
  m = __ockl_wfred_max_f32(m);
  if (m == -INFINITY) {  // every expert is off
    put_picks(a, t, lane, -1, 0.f);
    return;
  }
  // serr: bound of the error of a score.  Softmax: a score is off by its share of (|x - m| + 6 of
  // exp and products, EPL + 10 of the sum) 2^-24, s |x - m| at most 0.37 of the largest; sigmoid: by
  // (1 - s) (1.5 |x| + 2) + 3 of it, s (1 - s) |x| at most that of the largest logit if it is below -1, and
  // by all of it below 2^-126 (from |x| = 89 on: |x| of -128 and less does not matter, and may overflow).
  // What is off becomes -infinity: x 0 is NaN for it, and so is a NaN bias, and the larger of NaN and
  // -infinity is that.
  float sum = 1.f, serr;
  if (a.score == LC_MOE_SOFTMAX) {
    float e[EPL];
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      e[i] = exp_neg(x[i] - m);
      sum += e[i];
    }
    sum = __ockl_wfred_add_f32(sum);
    const float rs = 1.f / sum;
    serr = rs * (EPL + 17) * 0x1p-24f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = fmaxf(fmaf(x[i], 0.f, fmaf(e[i], rs, c[i])), -INFINITY);
  } else {
    const float top = 1.f / (1.f + __builtin_amdgcn_exp2f(m * -1.44269504f));
    serr = top * (8.f + 2.f * fminf(fmaxf(-m, 0.f), 128.f)) * 0x1p-24f + 0x1p-125f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x[i] * -1.44269504f));
      c[i] = fmaxf(fmaf(x[i], 0.f, s + c[i]), -INFINITY);
    }
  }

  bool whole = false;  // the token has to be taken in fp64
  if (a.top_groups < a.groups) {
    float* row = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int j = 0; j < EPL / V; ++j) {
      const int e = (j * 64 + lane) * V;
      if (e < a.E) {
        if constexpr (V == 4)
          *reinterpret_cast<float4*>(row + e) = make_float4(c[4 * j], c[4 * j + 1], c[4 * j + 2], c[4 * j + 3]);
        else
          row[e] = c[j];
      }
    }
    wave_fence();
    // 64 / (groups rounded up to a power of two) lanes a group
    const int sh = a.groups > 32 ? 0 : a.groups > 16 ? 1 : a.groups > 8 ? 2 : a.groups > 4 ? 3 : a.groups > 2 ? 4 : 5;
    const int g = lane >> sh, part = 1 << sh;
    float m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.groups) {
      const float* run = row + g * a.size;
      auto take = [&](float v) {
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      };
      if (a.size % 4 == 0) {
        for (int e = (lane & (part - 1)) * 4; e < a.size; e += part * 4) {
          const float4 q = *reinterpret_cast<const float4*>(run + e);
          take(q.x), take(q.y), take(q.z), take(q.w);
        }
      } else {
        for (int e = lane & (part - 1); e < a.size; e += part) take(run[e]);
      }
    }
    for (int o = 1; o < part; o <<= 1) {
      const float o1 = __shfl_xor(m1, o), o2 = __shfl_xor(m2, o);
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    }
    const bool two = a.rank == 2 && m2 > -INFINITY;
    const float best = two ? m1 + m2 : m1;
    int before = 0;  // groups ahead of the lane's, but for equal ones: if they make it too many, fp64 decides
    for (int j = 0; j < a.groups; ++j) before += lane_value(best, j << sh) > best ? 1 : 0;
    const bool kept = g < a.groups && before < a.top_groups;
    // half a step of every fp32 value that went into a group's score, and its scores' errors
    const float err = m1 > -INFINITY ? (two ? 2.f * serr + (fabsf(m1) + fabsf(m2) + fabsf(best)) * 0x1.1p-24f
                                            : serr + fabsf(m1) * 0x1.1p-24f) : 0.f;
    const float least = -__ockl_wfred_max_f32(kept || g >= a.groups ? -(kept ? best - err : INFINITY) : -INFINITY);
    const float most = __ockl_wfred_max_f32(kept || g >= a.groups ? -INFINITY : best + err);
    wave_fence();
    // (two biases near the largest float may overflow: fp64 then tells the groups apart)
    whole = (most > -INFINITY && !(least > most)) || __ballot(m1 > -INFINITY && !(fabsf(best) < INFINITY)) ||
            __popcll(__ballot(kept && m1 > -INFINITY)) > a.top_groups << sh;
    const unsigned long long live = __ballot(kept);
    const uint32_t magic = uint32_t((0x100000000ull + a.size - 1) / a.size);  // e / size, exact for e, size < 2^16
    auto keep = [&](int e) {
      const int ge = a.size == 1 ? e : int(__umulhi(uint32_t(e), magic));
      return e < a.E && (live >> ((ge << sh) & 63) & 1);
    };
    if (V == 4 && a.size % 4 == 0) {  // four experts of a lane are of one group
#pragma unroll
      for (int j = 0; j < EPL / V; ++j) {
        const bool in = keep((j * 64 + lane) * V);
#pragma unroll
        for (int i = 0; i < V; ++i) c[j * V + i] = in ? c[j * V + i] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = keep(((i / V) * 64 + lane) * V + i % V) ? c[i] : -INFINITY;
    }
  }

  // ---- what may be picked ----
  // A candidate is (c, expert, logit).
  float* g_c = reinterpret_cast<float*>(mine);
  int* g_e = reinterpret_cast<int*>(mine + 512);
  float* g_x = reinterpret_cast<float*>(mine + 768);
  float lm = c[0];  // the lane's largest
#pragma unroll
  for (int i = 1; i + 1 < EPL; i += 2) lm = fmaxf(lm, fmaxf(c[i], c[i + 1]));
  if constexpr (EPL % 2 == 0) lm = fmaxf(lm, c[EPL - 1]);
  int n = 65, place = 0;  // how many may be, and the place of the lane's first
  float bound = 0.f;
  for (int parts = EPL == 1 ? 1 : a.K <= 16 ? 16 : 64; !whole; parts = 64) {
    float kth = -INFINITY;
    if constexpr (EPL > 1) {
      int before = 0;
      float pm = lm;  // largest of the lane's part
      if (parts == 16) {
        pm = fmaxf(pm, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(pm), 0xB1, 0xF, 0xF, true)));  // lanes 1 0 3 2
        pm = fmaxf(pm, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(pm), 0x4E, 0xF, 0xF, true)));  // lanes 2 3 0 1
#pragma unroll
        for (int j = 0; j < 16; ++j) before += lane_value(pm, 4 * j) > pm ? 1 : 0;
      } else {
#pragma unroll 8
        for (int j = 0; j < 64; ++j) before += lane_value(pm, j) > pm ? 1 : 0;
      }
      kth = -__ockl_wfred_max_f32(before < a.K ? -pm : -INFINITY);
    }
    // (what is off is below every bound but one that overflows, of a bias near the lowest float: then all
    // 64 EPL places count, and the token is taken in fp64)
    bound = kth > -INFINITY ? kth - 2.f * serr - fabsf(kth) * 0x1p-22f : -__FLT_MAX__;
    int mine_n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) mine_n += c[i] >= bound ? 1 : 0;
    place = wave_scan(mine_n);
    n = __builtin_amdgcn_readlane(place, 63);
    place -= mine_n;
    if (n <= 64 || parts != 16) break;
  }
  if (n > 64) {
    select_token_f64(a, t, lane, reinterpret_cast<double*>(mine));
    return;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (c[i] >= bound) {
      g_c[place] = c[i];
      g_e[place] = ((i / V) * 64 + lane) * V + i % V;
      g_x[place] = x[i];
      ++place;
    }
  }
  wave_fence();
  float vc = lane < n ? g_c[lane] : -INFINITY, vx = g_x[lane];
  int ve = g_e[lane];
  wave_fence();
  // Sorted one k in lane k.
  auto put = [&](int place) {
    if (lane < n) {
      g_e[place] = ve;
      g_x[place] = vx;
    }
  };
  auto get = [&]() {
    wave_fence();
    ve = g_e[lane];
    vx = g_x[lane];
    wave_fence();
  };
  place = place_of(vc, n);
  const int was = ve;
  put(place);
  if (lane < n) g_c[place] = vc;
  wave_fence();
  // Where two are as good as equal, or equal (one place for both: one finds the other there), fp64
  // decides.  (The last lane has no next one; a place behind the last candidate does not count.)
  const float next = g_c[lane < 63 ? lane + 1 : 63], mine_c = g_c[lane];
  const bool near = lane < n && (g_e[place] != was || (lane < a.K && lane + 1 < n && mine_c - next <=
                                 2.f * serr + (fabsf(mine_c) + fabsf(next)) * 0x1.1p-24f));
  if (!__ballot(near)) {
    get();
  } else {
    wave_fence();
    double sum64 = 1.0;
    if (a.score == LC_MOE_SOFTMAX) {
      sum64 = 0.0;
#pragma unroll 1
      for (int e = lane; e < a.E; e += 64) {
        const float l = a.logits[size_t(t) * a.E + e];
        sum64 += l > -INFINITY ? exp(l - double(m)) : 0.0;
      }
      sum64 = wave_sum(sum64);
    }
    double c64 = 0.0;
    if (lane < n) {
      const double s = a.score == LC_MOE_SOFTMAX ? exp(vx - double(m)) / sum64 : 1.0 / (1.0 + exp(-double(vx)));
      c64 = s + (a.bias ? a.bias[ve] : 0.f);
    }
    put(place_of(c64, ve, n));
    get();
  }
  const bool valid = lane < n && lane < a.K;
  const float g = pick_gate(a, valid, valid ? vx : 0.f, m, sum);
  put_picks(a, t, lane, valid ? ve : -1, g);
}

// go(EPL, V) for a pool of E experts: how many of them a lane holds, and how many next to each other.
#define LCM_BY_POOL(E, go)        \
  do {                            \
    if ((E) % 4 == 0) {           \
      if ((E) <= 256) go(4, 4);   \
      else if ((E) <= 512) go(8, 4);   \
      else if ((E) <= 768) go(12, 4);  \
      else if ((E) <= 1024) go(16, 4); \
      else if ((E) <= 2048) go(32, 4); \
      else go(64, 4);             \
    } else {                      \
      if ((E) <= 64) go(1, 1);    \
      else if ((E) <= 128) go(2, 1);   \
      else if ((E) <= 256) go(4, 1);   \
      else if ((E) <= 512) go(8, 1);   \
      else if ((E) <= 1024) go(16, 1); \
      else if ((E) <= 2048) go(32, 1); \
      else go(64, 1);             \
    }                             \
  } while (0)

template <int EPL, int V>
static void select_launch(const SelectArgs& a, hipStream_t st) {
  // a wave's room: E fp64 scores (a token that is taken in fp64), or 64 candidates
  const int room = (a.E * 8 > 1024 ? a.E * 8 : 1024) + 15 & ~15;
  int waves = 4;
  while (waves > 1 && (waves * room > 32768 || (a.T + waves - 1) / waves < 256)) waves /= 2;
  select_kernel<EPL, V><<<dim3((a.T + waves - 1) / waves), dim3(waves * 64), waves * room, st>>>(a, room);
}

hipError_t launch_select(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits, const float* bias,
                         const uint8_t* mask, int32_t* idx, float* gate, hipStream_t st) {
  const int E = s.N + s.Z;
  const SelectArgs a{logits, bias, mask, idx, gate, s.T, E, s.K, g.score, g.groups, E / g.groups, g.top_groups,
                     g.group_rank, g.renorm != 0, g.scale};
#define LCM_GO(EPL, V) select_launch<EPL, V>(a, st)
  LCM_BY_POOL(E, LCM_GO);
#undef LCM_GO
  return hipGetLastError();
}

// ---- gradient ----------------------------------------------------------------------------

struct SelectBwArgs {
  const float* logits;
  const int32_t* idx;
  const float* dgate;
  const float* aux;
  float* dlogits;
  int T, E, K, score, renorm;
  float scale;
};

// One token by one wavefront, pick k in lane k, the row of logits or of dlogits_aux in registers
// (logit_row.h).  The picks' terms are put into a row of zeros in LDS.  Only the softmax without
// renorm needs every logit; the other forms read those of the picks, and what they take is the
// writing of dlogits and the reading of dlogits_aux.
template <int EPL, int V>
__global__ __launch_bounds__(256) void select_backward_kernel(SelectBwArgs a) {
  extern __shared__ __attribute__((aligned(16))) float rows[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * (blockDim.x >> 6) + wave;
  if (t >= a.T) return;
  float* dp = rows + size_t(wave) * ((a.E + 3) & ~3);
  const float* row = a.logits + size_t(t) * a.E;
  const int e = lane < a.K ? a.idx[size_t(t) * a.K + lane] : -1;
  float d[EPL];
  if (a.aux) {
    load_row<EPL, V>(a.aux + size_t(t) * a.E, a.E, lane, 0.f, d);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = 0.f;
  }
  const bool ok = static_cast<unsigned>(e) < static_cast<unsigned>(a.E);
  const float dg = ok ? a.dgate[size_t(t) * a.K + lane] : 0.f;
  const float x = ok ? row[e] : 0.f;
  if (!__ballot(ok)) {  // no pick, no gradient: the row is not read
    store_row<EPL, V>(a.dlogits + size_t(t) * a.E, a.E, lane, d);
    return;
  }
#pragma unroll
  for (int j = 0; j < EPL / V; ++j) {
    const int at = (j * 64 + lane) * V;
    if (at >= a.E) continue;
    if constexpr (V == 4) *reinterpret_cast<float4*>(dp + at) = make_float4(0.f, 0.f, 0.f, 0.f);
    else dp[at] = 0.f;
  }
  const bool whole = a.score == LC_MOE_SOFTMAX && !a.renorm;
  float v;  // the pick's own term
  if (a.renorm) {
    // the picks' shares, as in the forward
    const bool soft = a.score == LC_MOE_SOFTMAX, on = ok && x > -INFINITY;
    const float l = soft ? x : fminf(x, 0.f);
    const float top = __ockl_wfred_max_f32(on ? l : -INFINITY);
    float u = on ? exp_neg(l - top) : 0.f;
    const float s = 1.f / (1.f + exp_neg(-fabsf(x)));  // of the larger of s and 1 - s
    if (!soft) u *= s;
    const float sum = __ockl_wfred_add_f32(u);
    const float w = sum > 0.f ? u / sum : 0.f;
    // The shares sum to 1, so dg_k - sum w_j dg_j is a sum of differences, in which nothing cancels that is
    // not alike in dg itself: one pick, or gradients that are all the same, give 0.
    float rest = 0.f;
    for (int j = 0; j < a.K; ++j) rest = fmaf(lane_value(w, j), dg - lane_value(dg, j), rest);
    v = a.scale * (w * rest);
    if (!soft) v *= x > 0.f ? exp_neg(-x) * s : s;  // 1 - s
  } else if (a.score == LC_MOE_SIGMOID) {
    const float q = exp_neg(-fabsf(x)), s = 1.f / (1.f + q);
    v = a.scale * dg * (s * (q * s));
  } else {
    v = a.scale * dg;
  }
  // an index that repeats: its terms are added, in the order of the picks, and put once
  float sum_v = 0.f;
  bool again = false;
  for (int k = 0; k < a.K; ++k) {
    const int ek = __builtin_amdgcn_readlane(e, k);
    const float vk = lane_value(v, k);
    sum_v += ek == e ? vk : 0.f;
    again |= k < lane && ek == e;
  }
  wave_fence();
  if (ok && !again) dp[e] = sum_v;
  wave_fence();
  float m = 0.f, rs = 0.f, mean = 0.f;
  float p[EPL];
  if (whole) {
    load_row<EPL, V>(row, a.E, lane, -INFINITY, p);
    const RowSum r = softmax_row(p);
    m = r.m > -INFINITY ? r.m : 0.f;
    rs = r.sum > 0.f ? 1.f / r.sum : 0.f;
    mean = __ockl_wfred_add_f32(ok ? exp_neg(x - m) * rs * v : 0.f);
  }
#pragma unroll
  for (int j = 0; j < EPL / V; ++j) {
    const int at = (j * 64 + lane) * V;
    if (at >= a.E) continue;
    float q[V];
    if constexpr (V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(dp + at);
      q[0] = f.x, q[1] = f.y, q[2] = f.z, q[3] = f.w;
    } else {
      q[0] = dp[at];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[j * V + i] += whole ? p[j * V + i] * rs * (q[i] - mean) : q[i];
  }
  store_row<EPL, V>(a.dlogits + size_t(t) * a.E, a.E, lane, d);
}

template <int EPL, int V>
static void select_backward_launch(const SelectBwArgs& a, hipStream_t st) {
  const int room = ((a.E + 3) & ~3) * 4, waves = a.E <= 1024 ? 4 : 1;
  select_backward_kernel<EPL, V><<<dim3((a.T + waves - 1) / waves), dim3(waves * 64), waves * room, st>>>(a);
}

hipError_t launch_select_backward(const lc_moe_shape& s, const lc_moe_gating& g, const float* logits,
                                  const int32_t* idx, const float* dgate, const float* aux, float* dlogits,
                                  hipStream_t st) {
  const int E = s.N + s.Z;
  const SelectBwArgs a{logits, idx, dgate, aux, dlogits, s.T, E, s.K, g.score, g.renorm != 0, g.scale};
#define LCM_GO(EPL, V) select_backward_launch<EPL, V>(a, st)
  LCM_BY_POOL(E, LCM_GO);
#undef LCM_GO
  return hipGetLastError();
}

}  // namespace lcm
