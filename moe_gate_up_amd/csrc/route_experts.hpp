// Routing to experts by scores, with a bias for balance and groups of experts,
// and the gradient of the weights (the definitions are at
// moe_decode_route_experts in include/moe_decode.h).
//
// A row of up to 256 experts lies in 16 lanes (else in a whole wavefront): each
// group of experts in its own LG lanes, LG the largest power of two that the
// groups leave, so that a group's score is log2 LG DPP steps and a row's maximum
// 4 (or 6).  Each lane sorts its keys once; then every selection is the maximum of
// the lanes' first keys, and the lane that had it moves its others up.  Groups are taken
// alike before that.  Selection j lands in the row's lane j, which works out its weight.
//
// Choices are those of 64 bits.  Without a bias they go by the logits themselves.
// With one (or by sums of two scores) the FP32 values' errors are known; neighbours in the
// order of choice that lie nearer than those are compared in FP64, one exponential a
// lane, and a row that this does not settle (or whose groups are as near) is done again
// in FP64 by the whole wavefront at its end: about one row in 10000 of logits of 1.5 sigma.  Where more than eight experts
// beyond the choice lie within the error, all rows are: sigmoid scores that saturate and one bias for all, a softmax score
// that leaves the others nothing, logits of the type's lowest value beside others, a bias of -inf.  262144 tokens of 128
// experts, top-8, then take 520-640 us (47-53 otherwise), in groups with a bias of -inf 1040; 32 tokens 23-39 (3-4).
//
// Vector instructions bound it: 262144 tokens of 128 experts, FP32, sigmoid, bias, 8 groups, the two
// largest, top-8: 71-77 us for 151 MB (2.0 TB/s), 418 vector instructions for 4 rows, of them
// 96 quarters of an exponential or reciprocal, 120 for the 8 selections and 38 for the sort;
// in a graph 64-66.  Keys and numbers in two registers and a search for
// the lowest number each time took 188.  4 workgroups a CU that go on to the next rows,
// whose logits are requested ahead; one workgroup for 16 rows 93.  32 tokens of 256 experts: 5.4 us.
// The gradient: 41 us for 285 MB (6.9 TB/s, some of the logits from the memory-side cache).
#pragma once

#include "balance.hpp"
#include "quantize.hpp"

namespace moe {

constexpr int kScoreThreads = 256;
constexpr int kScoreWaves = kScoreThreads / 64;
// What decides on a row's experts: the logits (no bias), or softmax or sigmoid scores and a bias.
constexpr int kByLogit = 0, kBySoftmax = 1, kBySigmoid = 2;
constexpr int kScoreSigmoid = 1, kScoreRenorm = 2, kScoreTop2 = 4;

struct ScoreArgs {
  const float* bias;
  int32_t* ids;
  float* weights;
  long long ld;
  int T, E, k;
  int G, Eg, top;   // groups, experts of one, groups that are kept
  int lg;           // log2 of the lanes of one group
  int flags;
  float scale;
};

template <int LR>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, (uint32_t)dppi<0xB1>((int)v));
  v = max(v, (uint32_t)dppi<0x4E>((int)v));
  v = max(v, (uint32_t)dppi<0x141>((int)v));
  v = max(v, (uint32_t)dppi<0x140>((int)v));
  if constexpr (LR == 64) {
    v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    v = max(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}

// DPP move of a 64-bit value; lanes in rows outside ROW_MASK keep `old`.
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp64(double old, double v) {
  const uint64_t o = __builtin_bit_cast(uint64_t, old), s = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)s, CTRL, ROW_MASK, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(o >> 32), (int)(s >> 32), CTRL, ROW_MASK, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t s = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)s, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(s >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// f over the 64 lanes, in a fixed order; `none` leaves f's other operand as it is.
template <typename F>
__device__ __forceinline__ double wave_join_f64(double v, double none, F f) {
  v = f(v, dpp64<0xB1>(none, v));
  v = f(v, dpp64<0x4E>(none, v));
  v = f(v, dpp64<0x141>(none, v));
  v = f(v, dpp64<0x140>(none, v));
  v = f(v, dpp64<0x142, 0xA>(none, v));   // rows 1 and 3 get the rows below them
  v = f(v, dpp64<0x143, 0xC>(none, v));   // row 3 gets row 1's
  return last_lane(v);
}
__device__ __forceinline__ double wave_max_f64(double v) {
  return wave_join_f64(v, -__builtin_huge_val(), [](double a, double b) { return __builtin_fmax(a, b); });
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  return wave_join_f64(v, 0.0, [](double a, double b) { return a + b; });
}

// The selections of one row in FP64 by a wavefront: lane j < k gets the expert of
// selection j.  `c`: LDS for the row, of which every lane uses its own experts' places
// (lane, lane + 64, ...).
template <typename T>
__device__ __forceinline__ int select_row_f64(const T* row, const ScoreArgs& a, int lane, double* c) {
  constexpr double kInf = __builtin_huge_val(), kOut = __builtin_nan("");
  const bool sigmoid = a.flags & kScoreSigmoid, top2 = a.flags & kScoreTop2;
  double m = -kInf, sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double l = (double)elem_f32(row[e]);
    c[e] = l == l ? l : -kInf;   // -inf: ruled out
    m = c[e] > m ? c[e] : m;
  }
  m = wave_max_f64(m);
  m = m == -kInf ? 0.0 : m;
  auto power = [&](double l) { return exp(sigmoid ? -l : l - m); };
  if (!sigmoid) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) sum += power(c[e]);
    sum = wave_sum_f64(sum);
  }
  auto score = [&](double l) {
    const double p = power(l), s = sigmoid ? 1.0 / (1.0 + p) : p / sum;
    return l == -kInf || s != s ? -kInf : s;
  };
  if (a.bias) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const double v = score(c[e]) + (double)a.bias[e];
      c[e] = v == v ? v : -kInf;
    }
  }
  if (a.top < a.G) {
    double mine = -kInf;   // lane g: group g's score
#pragma unroll 1
    for (int g = 0; g < a.G; ++g) {
      double m1 = -kInf, m2 = -kInf;
      auto join = [&](double o) {
        const double low = o < m1 ? o : m1;
        m2 = low > m2 ? low : m2;
        m1 = o > m1 ? o : m1;
      };
#pragma unroll 1
      for (int e = g * a.Eg + ((lane - g * a.Eg) & 63); e < (g + 1) * a.Eg; e += 64)
        join(!a.bias && top2 ? score(c[e]) : c[e]);   // the largest score is the largest logit's
      // the largest, and the largest where its first lane shows its second
      const double top1 = wave_max_f64(m1);
      const uint64_t holds = __builtin_amdgcn_ballot_w64(m1 == top1);
      m2 = wave_max_f64(lane == (int)__builtin_ctzll(holds) ? m2 : m1);
      m1 = top1;
      mine = lane == g ? (top2 && m2 != -kInf ? m1 + m2 : m1) : mine;
    }
    uint64_t kept = 0;
    for (int i = 0; i < a.top; ++i) {
      const bool open = lane < a.G && !(kept >> lane & 1);
      const double best = wave_max_f64(open ? mine : -kInf);
      const uint64_t hit = __builtin_amdgcn_ballot_w64(open && mine == best);
      kept |= hit & (0 - hit);
    }
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64)
      if (!(kept >> (e / a.Eg) & 1)) c[e] = kOut;
  }
  int id = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = -kInf;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) best = c[e] > best ? c[e] : best;
    best = wave_max_f64(best);
    int at = 1 << 30;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) at = c[e] == best ? min(at, e) : at;
    at = 1024 - (int)wave_max_u32((uint32_t)(1024 - min(at, 1024)));   // the lowest
    id = lane == j ? at : id;
    if ((at & 63) == lane) c[at] = kOut;
  }
  return id;
}

// The lane's experts: V of its group's, in pieces of C, the group's lanes' pieces side by side.
template <int C>
__device__ __forceinline__ int score_in_group(int p, int v, int lg) {
  return (((v / C) << lg) + p) * C + v % C;
}

// V keys, the largest first (a merge-exchange network; every comparison is a maximum and a minimum).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = key[i + j], b = key[i + j + k];
            key[i + j] = max(a, b);
            key[i + j + k] = min(a, b);
          }
}

// Maximum and minimum over the row's lanes, which pass over NaN.  The moves have no value for lanes that they do not
// reach (there are none), so that they become operands of the maxima.
template <int CTRL>
__device__ __forceinline__ float dpp_any(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int LR, typename F>
__device__ __forceinline__ float row_join(float v, F f) {
  v = f(v, dpp_any<0xB1>(v));
  v = f(v, dpp_any<0x4E>(v));
  v = f(v, dpp_any<0x141>(v));
  v = f(v, dpp_any<0x140>(v));
  if constexpr (LR == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LR>
__device__ __forceinline__ float row_top(float v) {
  return row_join<LR>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LR>
__device__ __forceinline__ float row_low(float v) {
  return row_join<LR>(v, [](float a, float b) { return fminf(a, b); });
}

// e^x for x <= 0: 2^t with t = x log2 e rounded, and what the rounding left of the exponent in first order.
__device__ __forceinline__ float exp_below(float x) {
  const float t = x * 1.44269502f, e = __builtin_amdgcn_exp2f(t);
  const float v = __builtin_fmaf(e, __builtin_fmaf(t, -0.693147182f, x), e);
  return x < -100.0f ? 0.0f : v;   // also -inf, whose rest is NaN
}

// Renormalised sigmoid scores whose sum is less than this (all logits below -44) are quotients of e^(l - M) instead, M
// the largest of their logits: FP32 has no e^l below -87, but the quotients.  Down to M = -745, where 64 bits have
// no e^l either and the sum is 0.  Such rows are done again.
constexpr float kScoreSumSmall = 0x1p-64f, kScoreLogitNone = -745.13f;

// 1 / (1 + e^-l): a = e^-|l| cannot overflow.
__device__ __forceinline__ float sigmoid_exact(float l) {
  const float a = exp_below(-__builtin_fabsf(l));
  return (l >= 0.0f ? 1.0f : a) / (1.0f + a);
}

// Keys.  What decides (c: logit, or score + bias) becomes a whole number q of the row's range, of 32 - BITS bits,
// and 1024 (256) less the expert's number the bits below: one unsigned maximum finds the largest and of equals the
// lowest expert, and no two keys are alike.  0 is an expert out of play, q = 0 one that is ruled out; every other
// has q >= 1, since c is taken from the range's lower end first: -lo * unit + 1 would be rounded, to less than 1 as well.
template <typename T, int LR, int V, int C, int BY>
__global__ __launch_bounds__(kScoreThreads) void route_experts_kernel(const T* __restrict__ logits, ScoreArgs a) {
  constexpr int RW = 64 / LR;
  constexpr int BITS = LR == 16 ? 9 : 11;   // of the expert's number, 1 .. 256 or 1024
  constexpr float kTop = (float)((1u << (32 - BITS)) - 1u);   // of q
  constexpr float kInf = __builtin_huge_valf();
  __shared__ double lds[kScoreWaves][LR == 16 ? 256 : 1024];
  const int lane = threadIdx.x & 63, l = lane % LR;
  const int g = l >> a.lg, p = l & ((1 << a.lg) - 1);
  const int base = min(g, a.G - 1) * a.Eg;
  const int mine = g < a.G ? a.Eg : 0;   // a lane's last experts may be beyond the group's end, its lanes beyond the last group
  constexpr bool by_logit = BY == kByLogit;
  const bool sigmoid = BY == kBySigmoid || (by_logit && (a.flags & kScoreSigmoid));
  const bool renorm = a.flags & kScoreRenorm, top2 = a.flags & kScoreTop2, grouped = a.top < a.G;
  const bool slot = l < a.k;

  // What the lane's experts have for every row: the low bits of their keys (0: no such expert), and what -inf and no
  // expert are made NaN with: c = x * rule + x of logits, score + (x * 0 + rule) where rule is the bias less the smallest.
  uint32_t code[V];
  float rule[V], bias_hi = 0.0f, bias_lo = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int in = score_in_group<C>(p, v, a.lg);
    const float r = by_logit ? 0.0f : a.bias[base + min(in, a.Eg - 1)];
    code[v] = in < mine ? (uint32_t)(a.E - base - in) : 0u;
    rule[v] = in < mine ? r : qnan();
    bias_hi = v ? fmaxf(bias_hi, rule[v]) : rule[v];
    bias_lo = v ? fminf(bias_lo, rule[v]) : rule[v];
  }
  // scores lie in [0, 1]: with the bias, one range for all rows, whose lower end is 0
  const float least = row_low<LR>(bias_lo), score_hi = 1.0f + (row_top<LR>(bias_hi) - least);
  if constexpr (!by_logit) {
#pragma unroll
    for (int v = 0; v < V; ++v) rule[v] -= least;
  }

  // `sum`: of a softmax's exponentials; with renorm it becomes the selections'.
  auto weigh = [&](float logit, float m, float& sum, bool again) {
    float w;
    if (sigmoid) {
      w = sigmoid_exact(logit);
    } else {
      if (renorm) m = row_top<LR>(slot ? logit : -kInf);
      m = m == -kInf ? 0.0f : m;
      w = exp_below(logit - m);
    }
    w = slot ? w : 0.0f;
    if (renorm) {
      sum = row_sum<LR>(w);
      if (again && sigmoid && sum < kScoreSumSmall) {   // of the wavefront's one row
        m = row_top<LR>(slot ? logit : -kInf);
        w = slot && m > kScoreLogitNone ? exp_below(logit - m) : 0.0f;
        sum = row_sum<LR>(w);
      }
    }
    if (renorm || !sigmoid) w = sum == 0.0f ? 0.0f : w / sum;
    return w * a.scale;
  };
  constexpr int RAW = C == 1 ? V : V * (int)sizeof(T) / 4;
  auto request = [&](uint32_t (&raw)[RAW], int first) {   // a row's logits, of an expert that exists where the lane has none
    const T* row = logits + (long long)min(first + lane / LR, a.T - 1) * a.ld + base;
    if constexpr (C == 4) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const T* at = row + min(score_in_group<C>(p, v, a.lg), a.Eg - 4);
        if constexpr (sizeof(T) == 4) {
          const u32x4 q = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[v + i] = q.v[i];
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(at);
          raw[v / 2] = q.x;
          raw[v / 2 + 1] = q.y;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const T one = row[min(score_in_group<C>(p, v, a.lg), a.Eg - 1)];
        if constexpr (sizeof(T) == 4) raw[v] = __builtin_bit_cast(uint32_t, one);
        else raw[v] = one;
      }
    }
  };
  const int first0 = ((int)blockIdx.x * kScoreWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6))) * RW;
  const int step = (int)gridDim.x * kScoreWaves * RW;
  uint64_t again = 0;   // bit r % 64: a row of round r has to be done in FP64; its first id is -1
  uint32_t raw[RAW];
  request(raw, first0);
  for (int first = first0, round = 0; first < a.T; first += step, ++round) {
    const int t = min(first + lane / LR, a.T - 1);
    const T* row = logits + (long long)t * a.ld;
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (sizeof(T) == 4) x[v] = __builtin_bit_cast(float, raw[v]);
      else if constexpr (C == 4) x[v] = bf16_bits_f32((v & 1) ? raw[v / 2] >> 16 : raw[v / 2] & 0xFFFFu);
      else x[v] = bf16_bits_f32(raw[v]);
    }
    request(raw, first < a.T - step ? first + step : first);   // the next round's, or these again
    __builtin_amdgcn_sched_barrier(0);

    // the row's largest logit and its exponentials' sum, where the scores are a softmax
    float m = 0.0f, sum = 1.0f, inv = 1.0f;
    if (!sigmoid && (!by_logit || !renorm || (grouped && top2))) {
      m = -kInf;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] = code[v] ? x[v] : -kInf;
        m = fmaxf(m, x[v]);
      }
      m = row_top<LR>(m);
      m = m == -kInf ? 0.0f : m;
      sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += __builtin_amdgcn_exp2f((x[v] - m) * 1.44269504f);
      sum = row_sum<LR>(sum);
      inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    auto score = [&](float f) {   // of a logit less m (a sigmoid's is 0)
      return sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(f * -1.44269504f))
                     : __builtin_amdgcn_exp2f(f * 1.44269504f) * inv;
    };
    // A score in FP64, and whether one's choice lies above another's.  A softmax's sum is that of FP32, whose error both
    // have in common: 2^-18 of the scores' difference.
    auto score64 = [&](float f) {
      const double p = exp(sigmoid ? -(double)f : (double)f - (double)m);
      return sigmoid ? 1.0 / (1.0 + p) : p * (double)inv;
    };
    auto above = [&](double s1, float b1, double s2, float b2) {
      const double c1 = s1 + (double)b1, c2 = s2 + (double)b2;
      return c1 - c2 > 0x1p-48 * (1.0 + __builtin_fabs(c1)) + (sigmoid ? 0.0 : 0x1p-18 * __builtin_fabs(s1 - s2));
    };
    // Errors of FP32 scores.  Sigmoid: e^-l within (1.5 |l| + 2) 2^-24, and |l| s (1 - s) < 0.23, the reciprocal and the
    // sum of 1: 5 2^-24 in all.  Softmax: (|l - m| + 3) 2^-23 and the sum's 10 2^-23 of s, |l - m| s < 0.4 of the largest
    // score `inv`: 2^-19 inv.  Logits have none.
    const float err = by_logit ? 0.0f : sigmoid ? 5.0f * 0x1p-24f : 0x1p-19f * inv;

    // what decides, from the range's lower end; NaN: ruled out or no expert, which maxima and minima pass over
    float c[V], hi = score_hi, lo = 0.0f, hi_lane = 0.0f;
    if (by_logit) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = __builtin_fmaf(x[v], rule[v], x[v]);
        hi = v ? fmaxf(hi, c[v]) : c[v];
        lo = v ? fminf(lo, c[v]) : c[v];
      }
      hi_lane = hi;
      hi = row_top<LR>(hi);
      lo = row_low<LR>(lo);
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] -= lo;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = score(x[v] - m) + __builtin_fmaf(x[v], 0.0f, rule[v]);
    }
    // q = 1 + c * unit, truncated and cut off above: each step never goes down where the logit or score + bias goes up
    const float range = hi - lo;
    const float unit = range > 0x1p-100f && range < kInf ? (kTop - 4.0f) / range : 1.0f;
    // Two experts further apart than this are in order: both scores' errors; the biases' difference, up to range - 1, and
    // its sum with the score, up to range, round by 2^-24 of themselves for each; the product's rounding, the truncation.
    const uint32_t near =
        by_logit ? 4u : (uint32_t)fminf((2.0f * err + 0x1p-23f * (2.0f * range - 1.0f)) * unit + 3.0f, kTop);
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // the middle one of three; of a NaN and two numbers the smaller
      const float q = __builtin_amdgcn_fmed3f(__builtin_fmaf(c[v], unit, 1.0f), 0.0f, kTop);
      key[v] = (uint32_t)q << BITS | code[v];
    }
    // biases whose range is not a finite number go to 64 bits; of logits, not a number: all are ruled out
    bool doubt = !(range < kInf) && (!by_logit || range == range);
    sort_keys<V>(key);
    if (grouped) {
      uint32_t gk, last = 0;
      if (by_logit && !top2) {   // the largest score is the largest logit's: compared as they are, then by number
        float m1 = hi_lane;
        if (a.lg > 0) m1 = fmaxf(m1, dpp<0xB1>(m1));
        if (a.lg > 1) m1 = fmaxf(m1, dpp<0x4E>(m1));
        if (a.lg > 2) m1 = fmaxf(m1, dpp<0x141>(m1));
        if (a.lg > 3) m1 = fmaxf(m1, dpp<0x140>(m1));
        if constexpr (LR == 64) {
          if (a.lg > 4) m1 = fmaxf(m1, __shfl_xor(m1, 16));   // 64 lanes are one group
        }
        gk = g < a.G ? route_key(m1 == m1 ? m1 : -kInf) : 0u;
        for (int i = 0; i < a.top; ++i) {
          last = row_max_u32<LR>(gk);
          const uint32_t at = row_max_u32<LR>(gk == last ? (uint32_t)(64 - g) : 0u);
          gk = (uint32_t)(64 - g) == at ? 0u : gk;
        }
      } else {
        uint32_t k1 = key[0], k2 = key[1];   // the group's two largest
        auto join = [&](uint32_t o1, uint32_t o2) {
          k2 = max(min(k1, o1), max(k2, o2));
          k1 = max(k1, o1);
        };
        if (a.lg > 0) join((uint32_t)dppi<0xB1>((int)k1), (uint32_t)dppi<0xB1>((int)k2));
        if (a.lg > 1) join((uint32_t)dppi<0x4E>((int)k1), (uint32_t)dppi<0x4E>((int)k2));
        if (a.lg > 2) join((uint32_t)dppi<0x141>((int)k1), (uint32_t)dppi<0x141>((int)k2));
        if (a.lg > 3) join((uint32_t)dppi<0x140>((int)k1), (uint32_t)dppi<0x140>((int)k2));
        if constexpr (LR == 64) {
          if (a.lg > 4) join((uint32_t)__shfl_xor((int)k1, 16), (uint32_t)__shfl_xor((int)k2, 16));
        }
        // the group's score in whole numbers, then its number, so that no two are alike
        const uint32_t q1 = k1 >> BITS, q2 = k2 >> BITS;
        uint32_t s = q1, within = near;
        if (top2) {
          doubt |= g < a.G && q1 != 0u && q2 == 0u;   // one alone is left: not a sum of two
          s = (q1 + q2) >> 1;
          within = near + 2u;
          if (by_logit) {   // of the scores, whose order the logits' is; a logit less m is known to 5 units
            const float back = 1.0f / unit, l1 = lo - m + (float)(q1 - 1u) * back, l2 = lo - m + (float)(q2 - 1u) * back;
            const float e = (sigmoid ? 0x1p-21f : 0x1p-19f * inv) + 10.0f * back * (sigmoid ? 0.25f : inv) + 0x1p-22f;
            s = q1 ? 1u + (uint32_t)fminf((score(l1) + score(l2)) * (0.5f * (kTop - 4.0f)), kTop) : 0u;
            within = (uint32_t)fminf(2.0f * e * kTop + 4.0f, kTop);
          }
        }
        gk = g < a.G ? s << 7 | (uint32_t)(64 - g) : 0u;
        for (int i = 0; i < a.top; ++i) {
          last = row_max_u32<LR>(gk);
          gk = gk == last ? 0u : gk;
        }
        const uint32_t out = row_max_u32<LR>(gk) >> 7, in = last >> 7;
        doubt |= in != 0u && in - out <= within;
      }
      key[0] = g < a.G && gk == 0u ? key[0] : 0u;   // a lane that is out shows nothing
    }
    uint32_t got = 0;
    auto pop = [&](uint32_t M) {   // M's lane goes on to its next
      const bool won = key[0] == M;
#pragma unroll
      for (int v = 0; v + 1 < V; ++v) key[v] = won ? key[v + 1] : key[v];
      key[V - 1] = won ? 0u : key[V - 1];
    };
    for (int j = 0; j < a.k; ++j) {
      const uint32_t M = row_max_u32<LR>(key[0]);
      got = l == j ? M : got;
      pop(M);
    }
    constexpr uint32_t kLow = (1u << BITS) - 1u;
    int id = slot ? a.E - (int)(got & kLow) : 0;
    float logit = slot ? elem_f32(row[id]) : 0.0f;
    const float bias = !by_logit && slot ? a.bias[id] : 0.0f;
    {   // neighbours in order of choice
      const uint32_t q = got >> BITS, q2 = (uint32_t)__shfl_down((int)got, 1) >> BITS;
      const float l2 = __shfl_down(logit, 1), b2 = __shfl_down(bias, 1);
      bool unsure = l + 1 < a.k && !(q == 0u || q - q2 > near || (by_logit ? logit >= l2 : logit == l2 && bias == b2));
      if (!by_logit && __builtin_amdgcn_ballot_w64(unsure)) {
        const double s = score64(logit), s2 = __shfl_down(s, 1);
        unsure = unsure && !above(s, bias, s2, b2);
      }
      doubt |= unsure;
    }
    // the first that was not taken, and all that are as near
    const int last_slot = (lane & ~(LR - 1)) + a.k - 1;
    const uint32_t qk = (uint32_t)__shfl((int)got, last_slot) >> BITS;
    uint32_t M = row_max_u32<LR>(key[0]);
    bool close = M >> BITS && qk - (M >> BITS) <= near;
    if (__builtin_amdgcn_ballot_w64(close)) {
      const float lk = __shfl(logit, last_slot), bk = __shfl(bias, last_slot);
      const double sk = by_logit ? 0.0 : score64(lk);
      for (int i = 0; __builtin_amdgcn_ballot_w64(close); ++i) {
        const int e = close ? a.E - (int)(M & kLow) : 0;
        const float le = elem_f32(row[e]), be = by_logit ? 0.0f : a.bias[e];
        doubt |= close && (i >= 8 || !(by_logit ? lk >= le : (lk == le && bk == be) || above(sk, bk, score64(le), be)));
        pop(M);   // a row without one more to look at comes to nothing here, and is not looked at again
        M = row_max_u32<LR>(key[0]);
        close = close && !doubt && M >> BITS && qk - (M >> BITS) <= near;
      }
    }
    const float w = weigh(logit, m, sum, false);
    doubt |= sigmoid && renorm && slot && sum < kScoreSumSmall && logit > kScoreLogitNone;
    doubt = row_max_u32<LR>(doubt ? 1u : 0u) != 0u;
    if (__builtin_amdgcn_ballot_w64(doubt)) again |= 1ull << (round & 63);
    if (slot && first + lane / LR < a.T) {
      a.ids[(long long)t * a.k + l] = doubt && l == 0 ? -1 : id;
      a.weights[(long long)t * a.k + l] = w;
    }
  }
  if (!again) return;
  for (int first = first0, round = 0; first < a.T; first += step, ++round) {
    if (!(again >> (round & 63) & 1)) continue;
    for (int t = first; t < min(first + RW, a.T); ++t) {
      int32_t* ids = a.ids + (long long)t * a.k;
      // read by the lane that wrote it
      const int mark = lane == (t - first) * LR ? ids[0] : 0;
      if (!__builtin_amdgcn_ballot_w64(mark < 0)) continue;
      const T* row = logits + (long long)t * a.ld;
      const int sel = select_row_f64(row, a, lane, lds[threadIdx.x >> 6]);
      const int id = __shfl(sel, l);
      float m = 0.0f, sum = 1.0f;
      if (!sigmoid && !renorm) {
        m = -kInf;
        for (int e = l; e < a.E; e += LR) m = fmaxf(m, elem_f32(row[e]));
        m = row_max<LR>(m);
        m = m == -kInf ? 0.0f : m;
        sum = 0.0f;
        for (int e = l; e < a.E; e += LR) sum += exp_below(elem_f32(row[e]) - m);
        sum = row_sum<LR>(sum);
      }
      const float w = weigh(slot ? elem_f32(row[id]) : 0.0f, m, sum, true);
      if (slot && lane < LR) {
        ids[l] = id;
        a.weights[(long long)t * a.k + l] = w;
      }
    }
  }
}

// The gradient of the weights.  The k chosen experts' terms are scattered into the
// row in LDS (added, so that an expert that stands there twice gets both) and the
// row is written from there.  Only a softmax that is not renormalised needs the other logits.
template <typename T, int LR, int V, int C>
__global__ __launch_bounds__(kScoreThreads) void route_experts_backward_kernel(
    const T* __restrict__ logits, long long ld, const int32_t* __restrict__ ids, const float* __restrict__ grad,
    T* __restrict__ d, long long ld_d, int rows, int E, int k, int flags, float scale) {
  constexpr int RW = 64 / LR, kCols = LR * V;
  constexpr float kInf = __builtin_huge_valf();
  __shared__ __attribute__((aligned(16))) float lds[kScoreWaves][RW][kCols];
  const int lane = threadIdx.x & 63, l = lane % LR, w = threadIdx.x >> 6;
  const int t0 = ((int)blockIdx.x * kScoreWaves + w) * RW + lane / LR;
  const int t = min(t0, rows - 1);
  const T* row = logits + (long long)t * ld;
  float* mine = lds[w][lane / LR];
  const bool sigmoid = flags & kScoreSigmoid, renorm = flags & kScoreRenorm, dense = !sigmoid && !renorm;
#pragma unroll
  for (int v = 0; v < V; ++v) mine[balance_col<LR, C>(l, v)] = 0.0f;

  float x[V], inv = 0.0f, m = 0.0f;
  if (dense) {   // exponentials relative to the largest logit m; a row's lowest values may swallow a logsumexp's logarithm
    RowLoad<T, LR, V, C> r;
    r.load(row, E, l);
    r.values(x, E, l, true);
    m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = row_max<LR>(m);
    m = m == -kInf ? 0.0f : m;
    row_softmax<LR, V>(x, inv);
  }
  const int id = l < k ? ids[(long long)t * k + l] : -1;
  const bool slot = (unsigned)id < (unsigned)E;
  const float g = slot ? grad[(long long)t * k + l] * scale : 0.0f;
  const float logit = slot ? elem_f32(row[id]) : -kInf;
  float term, dot = 0.0f;
  if (dense) {
    const float s = slot ? expf(logit - m) * inv : 0.0f;
    dot = row_sum<LR>(slot ? g * s : 0.0f);
    term = g;
  } else {
    float s, rest = 1.0f;   // rest: 1 - s, without the cancellation
    if (sigmoid) {
      s = slot ? 1.0f / (1.0f + expf(-logit)) : 0.0f;
      rest = 1.0f / (1.0f + expf(logit));
    } else {
      m = row_max<LR>(logit);
      m = m == -kInf ? 0.0f : m;
      s = slot ? expf(logit - m) : 0.0f;
    }
    if (renorm) {
      float sum = row_sum<LR>(s);
      const bool small = sigmoid && sum < kScoreSumSmall;
      if (__builtin_amdgcn_ballot_w64(small)) {
        m = row_max<LR>(logit);
        s = !small ? s : m > kScoreLogitNone ? expf(logit - m) : 0.0f;
        sum = row_sum<LR>(s);
      }
      s = sum == 0.0f ? 0.0f : s / sum;
      dot = row_sum<LR>(slot ? g * s : 0.0f);
    }
    term = s * rest * (g - dot);
  }
  __syncthreads();
  if (slot) atomicAdd(&mine[id], term);
  __syncthreads();
  if (t0 >= rows) return;
  T* out = d + (long long)t * ld_d;
  float f[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f[v] = mine[balance_col<LR, C>(l, v)];
    if (dense) f[v] = x[v] * inv * (f[v] - dot);
  }
#pragma unroll
  for (int v = 0; v < V; v += C) {
    const int c = balance_col<LR, C>(l, v);
    if (c >= E) continue;
    if constexpr (C == 4) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32_quad*>(out + c) = f32_quad{f[v], f[v + 1], f[v + 2], f[v + 3]};
      } else {
        *reinterpret_cast<u32_pair*>(out + c) =
            u32_pair{(uint32_t)f32_to_bf16_rne(f[v]) | (uint32_t)f32_to_bf16_rne(f[v + 1]) << 16,
                     (uint32_t)f32_to_bf16_rne(f[v + 2]) | (uint32_t)f32_to_bf16_rne(f[v + 3]) << 16};
      }
    } else {
      if constexpr (sizeof(T) == 4) out[c] = f[v];
      else out[c] = f32_to_bf16_rne(f[v]);
    }
  }
}

}  // namespace moe
