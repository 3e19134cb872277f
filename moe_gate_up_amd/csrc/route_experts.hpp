// Routing to experts by scores, with a bias for balance and groups of experts,
// and the gradient of the weights (the definitions are at
// moe_decode_route_experts in include/moe_decode.h).
//
// A row of up to 256 experts lies in 16 lanes (else in a whole wavefront): each
// group of experts in its own LG lanes, LG the largest power of two that the
// groups leave, so that a group's score is log2 LG DPP steps and a row's maximum
// 4 (or 6).  The groups are taken one by one, then the experts: the maximum of the
// order-preserving keys in play, the lowest expert that holds it, and that key out
// of play.  Selection j lands in the row's lane j, which works out its weight.
//
// Choices are those of 64 bits.  Without a bias they go by the logits themselves.
// With one (or by sums of two scores) the FP32 values' errors are known, and a row
// in which two of them that the choice hangs on lie nearer than that is done again
// in FP64 by the whole wavefront (one row in some hundreds).
#pragma once

#include "balance.hpp"
#include "quantize.hpp"

namespace moe {

constexpr int kScoreThreads = 256;
constexpr int kScoreWaves = kScoreThreads / 64;
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

// A score's key: a NaN ranks with -inf, whose key is above 0 (out of play).
__device__ __forceinline__ uint32_t score_key(float c) { return route_key(c == c ? c : -__builtin_huge_valf()); }

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const double t = __shfl_xor(v, o);
    v = t > v ? t : v;
  }
  return v;
}

__device__ __forceinline__ int wave_min_i32(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = min(v, __shfl_xor(v, o));
  return v;
}

// The selections of one row in FP64 by a wavefront, of up to 64 NV experts: lane
// j < k gets the expert of selection j.
template <typename T, int NV>
__device__ __noinline__ int select_row_f64(const T* row, const ScoreArgs& a, int lane) {
  constexpr double kInf = __builtin_huge_val();
  double c[NV];     // what decides; -inf: ruled out
  double own[NV];   // what the groups' scores are of
  double m = -kInf;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = 64 * v + lane;
    const double l = e < a.E ? (double)elem_f32(row[min(e, a.E - 1)]) : -kInf;
    c[v] = l == l ? l : -kInf;
    m = c[v] > m ? c[v] : m;
  }
  m = wave_max_f64(m);
  m = m == -kInf ? 0.0 : m;
  const bool sigmoid = a.flags & kScoreSigmoid;
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    own[v] = sigmoid ? 1.0 / (1.0 + exp(-c[v])) : exp(c[v] - m);
    sum += own[v];
  }
  if (!sigmoid) {
    sum = wave_sum(sum);
#pragma unroll
    for (int v = 0; v < NV; ++v) own[v] /= sum;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = 64 * v + lane;
    const bool out = c[v] == -kInf;
    if (a.bias) {
      own[v] += (double)a.bias[min(e, a.E - 1)];
      own[v] = own[v] == own[v] ? own[v] : -kInf;
      c[v] = out ? -kInf : own[v];
    }
    own[v] = out ? -kInf : own[v];
    if (!a.bias && !(a.flags & kScoreTop2)) own[v] = c[v];   // the largest score is the largest logit's
  }
  uint64_t kept = ~0ull;
  if (a.top < a.G) {
    double mine = -kInf;   // lane g: group g's score
    for (int g = 0; g < a.G; ++g) {
      double m1 = -kInf;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = 64 * v + lane;
        m1 = e >= g * a.Eg && e < (g + 1) * a.Eg && own[v] > m1 ? own[v] : m1;
      }
      m1 = wave_max_f64(m1);
      double score = m1;
      if ((a.flags & kScoreTop2) && m1 != -kInf) {
        int at = 1 << 30;
#pragma unroll
        for (int v = NV - 1; v >= 0; --v) {
          const int e = 64 * v + lane;
          at = e >= g * a.Eg && e < (g + 1) * a.Eg && own[v] == m1 ? e : at;
        }
        at = wave_min_i32(at);
        double m2 = -kInf;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = 64 * v + lane;
          m2 = e >= g * a.Eg && e < (g + 1) * a.Eg && e != at && own[v] > m2 ? own[v] : m2;
        }
        m2 = wave_max_f64(m2);
        score = m2 == -kInf ? m1 : m1 + m2;
      }
      mine = lane == g ? score : mine;
    }
    kept = 0;
    for (int i = 0; i < a.top; ++i) {
      const bool open = lane < a.G && !(kept >> lane & 1);
      const double best = wave_max_f64(open ? mine : -kInf);
      const uint64_t hit = __builtin_amdgcn_ballot_w64(open && mine == best);
      kept |= hit & (0 - hit);
    }
  }
  uint32_t open = 0;   // bit v: expert 64 v + lane is in play
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = 64 * v + lane;
    open |= e < a.E && (kept >> (e / a.Eg) & 1) ? 1u << v : 0u;
  }
  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = -kInf;
#pragma unroll
    for (int v = 0; v < NV; ++v) best = (open >> v & 1) && c[v] > best ? c[v] : best;
    best = wave_max_f64(best);
    int at = 1 << 30;
#pragma unroll
    for (int v = NV - 1; v >= 0; --v) at = (open >> v & 1) && c[v] == best ? 64 * v + lane : at;
    at = wave_min_i32(at);
    id = lane == j ? at : id;
#pragma unroll
    for (int v = 0; v < NV; ++v) open &= at == 64 * v + lane ? ~(1u << v) : ~0u;
  }
  return id;
}

// The lane's experts: V of its group's, in pieces of C, the group's lanes' pieces side by side.
template <int C>
__device__ __forceinline__ int score_in_group(int p, int v, int lg) {
  return (((v / C) << lg) + p) * C + v % C;
}

template <typename T, int LR, int V, int C>
__global__ __launch_bounds__(kScoreThreads) void route_experts_kernel(const T* __restrict__ logits, ScoreArgs a) {
  constexpr int RW = 64 / LR;
  constexpr float kInf = __builtin_huge_valf();
  const int lane = threadIdx.x & 63, l = lane % LR;
  const int first = ((int)blockIdx.x * kScoreWaves + (int)(threadIdx.x >> 6)) * RW;   // this wavefront's rows
  if (first >= a.T) return;
  const int t = min(first + lane / LR, a.T - 1);
  const T* row = logits + (long long)t * a.ld;
  const int g = l >> a.lg, p = l & ((1 << a.lg) - 1);
  const int base = min(g, a.G - 1) * a.Eg;

  float x[V];
  if constexpr (C == 4) {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const T* at = row + base + min(score_in_group<C>(p, v, a.lg), a.Eg - 4);
      if constexpr (sizeof(T) == 4) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v + i] = __builtin_bit_cast(float, q.v[i]);
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(at);
        x[v] = bf16_bits_f32(q.x & 0xFFFFu);
        x[v + 1] = bf16_bits_f32(q.x >> 16);
        x[v + 2] = bf16_bits_f32(q.y & 0xFFFFu);
        x[v + 3] = bf16_bits_f32(q.y >> 16);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = elem_f32(row[base + min(score_in_group<C>(p, v, a.lg), a.Eg - 1)]);
  }
  // a lane's last experts may be beyond the group's end, its lanes beyond the last group
  const int mine = g < a.G ? a.Eg : 0;
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = score_in_group<C>(p, v, a.lg) < mine && x[v] == x[v] ? x[v] : -kInf;

  const bool sigmoid = a.flags & kScoreSigmoid, renorm = a.flags & kScoreRenorm, top2 = a.flags & kScoreTop2;
  const bool grouped = a.top < a.G;
  // the row's largest logit and its exponentials' sum, where the scores are a softmax
  float m = 0.0f, sum = 1.0f, inv = 1.0f;
  if (!sigmoid && (a.bias || !renorm || (grouped && top2))) {
    m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = row_max<LR>(m);
    m = m == -kInf ? 0.0f : m;
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += __builtin_amdgcn_exp2f((x[v] - m) * 1.44269504f);
    sum = row_sum<LR>(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  auto score = [&](float f) {
    return sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(f * -1.44269504f))
                   : __builtin_amdgcn_exp2f((f - m) * 1.44269504f) * inv;
  };
  // Errors of FP32 scores.  Sigmoid: e^-l within (1.5 |l| + 2) 2^-24, and |l| s (1 - s) < 0.23, the reciprocal and the
  // sum of 1: 5 2^-24 in all.  Softmax: (|l - m| + 3) 2^-23 and the sum's 10 2^-23 of s, |l - m| s < 0.4 of the largest
  // score `inv`: 2^-19 inv.  A bias's sum rounds by 2^-24 |c|.  Two choices further apart than `near` are in order; a
  // group's score is the sum of two.
  const float by_score = sigmoid ? 0x1p-20f : 0x1p-18f * inv;
  auto near = [&](float c) { return by_score + 0x1p-22f * __builtin_fabsf(c); };

  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int in = score_in_group<C>(p, v, a.lg);
    const float c = a.bias ? (x[v] == -kInf ? -kInf : score(x[v]) + a.bias[base + min(in, a.Eg - 1)]) : x[v];
    key[v] = in < mine ? score_key(c) : 0u;
  }
  bool doubt = false;
  if (grouped) {
    const bool by_logit = !a.bias && !top2;   // the largest score is the largest logit's
    float m1 = -kInf, m2 = -kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float c = key[v] ? route_key_value(key[v]) : -kInf;
      if (!a.bias && top2) c = c == -kInf ? c : score(c);
      m2 = fmaxf(m2, fminf(m1, c));
      m1 = fmaxf(m1, c);
    }
    auto join = [&](float o1, float o2) {
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    };
    if (a.lg > 0) join(dpp<0xB1>(m1), dpp<0xB1>(m2));
    if (a.lg > 1) join(dpp<0x4E>(m1), dpp<0x4E>(m2));
    if (a.lg > 2) join(dpp<0x141>(m1), dpp<0x141>(m2));
    if (a.lg > 3) join(dpp<0x140>(m1), dpp<0x140>(m2));
    if constexpr (LR == 64) {
      if (a.lg > 4) join(__shfl_xor(m1, 16), __shfl_xor(m2, 16));   // 64 lanes are one group: not grouped
    }
    const float s = top2 && m2 != -kInf ? m1 + m2 : m1;
    uint32_t gk = g < a.G ? score_key(s) : 0u, last = 0;
    for (int i = 0; i < a.top; ++i) {
      last = row_max_u32<LR>(gk);
      const uint32_t at = 64u - row_max_u32<LR>(gk == last ? 64u - (uint32_t)g : 0u);
      gk = (uint32_t)g == at ? 0u : gk;
    }
    const bool kept = g < a.G && gk == 0u;
    if (!by_logit) {
      const float in = route_key_value(last), out = route_key_value(row_max_u32<LR>(gk));
      doubt = in != -kInf && !(in - out > 4.0f * near(__builtin_fabsf(in) + __builtin_fabsf(out)));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = kept ? key[v] : 0u;
  }
  int id = 0;
  uint32_t got = 0, next = 0;
  for (int j = 0; j <= a.k; ++j) {
    uint32_t M = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) M = max(M, key[v]);
    M = row_max_u32<LR>(M);
    next = M;
    if (j == a.k) break;
    uint32_t at = 0;   // 1024 less the lowest expert that holds it
#pragma unroll
    for (int v = 0; v < V; ++v)
      at = max(at, key[v] == M ? 1024u - (uint32_t)(base + score_in_group<C>(p, v, a.lg)) : 0u);
    at = 1024u - row_max_u32<LR>(at);
    if (l == j) {
      id = (int)at;
      got = M;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = at == (uint32_t)(base + score_in_group<C>(p, v, a.lg)) ? 0u : key[v];
  }
  const bool slot = l < a.k;
  float logit = route_key_value(got);
  if (a.bias) {
    logit = slot ? elem_f32(row[id]) : 0.0f;
    const float b = slot ? a.bias[id] : 0.0f;
    const uint32_t below = (uint32_t)__shfl_down((int)got, 1);   // by all lanes: one that is idle gives nothing
    const uint32_t behind = l == a.k - 1 ? next : below;
    const float logit2 = __shfl_down(logit, 1), b2 = __shfl_down(b, 1);
    const float c = route_key_value(got), c2 = route_key_value(behind);
    const bool sure = behind == 0u || c == -kInf || c - c2 > near(c) || (l < a.k - 1 && logit == logit2 && b == b2);
    doubt |= slot && !sure;
  }
  uint64_t again = __builtin_amdgcn_ballot_w64(doubt);
  if (again) {
    for (int r = 0; r < RW; ++r) {
      if (!(again >> (r * LR) & (LR == 64 ? ~0ull : 0xFFFFull))) continue;
      const int tr = min(first + r, a.T - 1);
      const T* from = logits + (long long)tr * a.ld;
      const int sel = select_row_f64<T, LR == 16 ? 4 : 16>(from, a, lane);
      const int moved = __shfl(sel, l);
      if (lane / LR == r) {
        id = moved;
        logit = slot ? elem_f32(from[id]) : 0.0f;
      }
    }
  }
  float w;
  if (sigmoid) {
    w = 1.0f / (1.0f + expf(-logit));
  } else {
    if (renorm) m = row_max<LR>(slot ? logit : -kInf);
    m = m == -kInf ? 0.0f : m;
    w = expf(logit - m);
  }
  w = slot ? w : 0.0f;
  if (renorm) sum = row_sum<LR>(w);
  if (renorm || !sigmoid) w = sum == 0.0f ? 0.0f : w / sum;
  if (slot && first + lane / LR < a.T) {
    a.ids[(long long)t * a.k + l] = id;
    a.weights[(long long)t * a.k + l] = w * a.scale;
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
      const float sum = row_sum<LR>(s);
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
