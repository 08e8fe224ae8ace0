// Routing to experts: each token's k experts and their weights from the router's logits, and the gradient
// for the logits.  Bound by memory (the logits once, 8 k bytes out) or, in a decode step, by the launch.
//
// A row of logits belongs to LPR lanes of one wave, V = J W values each in registers (W to a 16-byte load,
// element (j LPR + lane) W + i), so nothing but a row's own lanes meets and no barrier is needed.
#include "block_ops.h"
#include "block_sizes.h"
#include "mm_common.h"
#include "wave_ops.h"

#include <math.h>

#include <type_traits>

namespace gmlp {

constexpr int RT = 256;      // threads of a workgroup

// ----------------------------------------------------------------------------- logits
template <int TYPE>
struct Logit {
  using T = uint16_t;
  static constexpr int W = 8;
  static __device__ __forceinline__ float up(uint16_t v) { return Elem<TYPE>::up(v); }
  static __device__ __forceinline__ uint16_t down(float f) { return Elem<TYPE>::down(f); }
};
template <>
struct Logit<ROUTE_FP32> {
  using T = float;
  static constexpr int W = 4;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float f) { return f; }
};
constexpr float kMasked = -INFINITY;

// The lane's values of a row, kMasked behind the last expert (the hardware takes any alignment).
template <int TYPE, int LPR, int J>
__device__ __forceinline__ void load_row(const typename Logit<TYPE>::T* row, int E, int lane, float* l) {
  using L = Logit<TYPE>;
  constexpr int W = L::W;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e0 = (j * LPR + lane) * W;
    typename L::T t[W];
    if (e0 + W <= E) {
      __builtin_memcpy(t, row + e0, 16);
#pragma unroll
      for (int i = 0; i < W; ++i) l[j * W + i] = L::up(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) l[j * W + i] = e0 + i < E ? L::up(row[e0 + i]) : kMasked;
    }
  }
}
template <int LPR, int W>
__device__ __forceinline__ int expert_of(int v, int lane) { return (v / W * LPR + lane) * W + v % W; }

// ----------------------------------------------------------------------------- order
// Keys that compare as the numbers do, without a sign: 0 for a masked expert, the largest for NaN.
__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) return ~0u;
  const uint32_t u = __float_as_uint(f + 0.0f);               // -0 as +0
  return f == kMasked ? 0u : (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double d) {
  if (d != d) return ~0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
  return d == -INFINITY ? 0ull : (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double value_of(uint64_t key) {
  return __longlong_as_double((long long)((key >> 63) ? key & ~(1ull << 63) : ~key));
}

// The row's scores in 64 bits, whose sums with the bias are compared.
template <int LPR, int V>
__device__ __forceinline__ void scores64(const float* l, float top, bool sigmoid, double* s) {
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = sigmoid ? 1.0 / (1.0 + exp(-(double)l[v])) : exp((double)l[v] - (double)top);
    if (l[v] == kMasked) s[v] = 0.0;
    sum += s[v];
  }
  if (sigmoid) return;
  sum = lanes_sum<LPR>(sum);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] /= sum;
}

// The k experts of a row in order into sel (LDS, -1: none), in exact order: keys of 64 bits, from the
// logits or from scores in 64 bits.
template <int LPR, int J, int W>
__device__ void select_exact(const RouteArgs& p, const float* l, float top, int lane, uint64_t* keys, uint64_t* group_key,
                             int32_t* sel) {
  constexpr int V = J * W;
  uint64_t key[V], wide[V];
  const bool need = p.bias || (p.groups > 1 && p.group_best > 1);
  if (need) {
    double s[V];
    scores64<LPR, V>(l, top, p.sigmoid, s);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LPR, W>(v, lane);
      const double c = p.bias && e < p.E ? s[v] + (double)p.bias[e] : s[v];
      wide[v] = l[v] == kMasked ? 0ull : key_of(c);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!need) wide[v] = (uint64_t)key_of(l[v]) << 32;
    key[v] = p.bias ? wide[v] : (uint64_t)key_of(l[v]) << 32;
  }
  if (p.groups > 1) {
    const int per = p.E / p.groups;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LPR, W>(v, lane);
      if (e < p.E) keys[e] = wide[v];
    }
    wave_fence();
    for (int g = lane; g < p.groups; g += LPR) {
      uint64_t a = 0, b = 0;                                   // the two largest
      for (int i = 0; i < per; ++i) {
        const uint64_t x = keys[g * per + i];
        b = x > a ? a : x > b ? x : b;
        a = x > a ? x : a;
      }
      if (p.group_best > 1 && b && a != ~0ull) a = b == ~0ull ? b : key_of(value_of(a) + value_of(b));
      group_key[g] = a;
    }
    wave_fence();
    for (int g = lane; g < p.groups; g += LPR) {
      const uint64_t mine = group_key[g];
      int better = 0;
      for (int o = 0; o < p.groups; ++o) {
        const uint64_t x = group_key[o];
        better += x > mine || (x == mine && o < g);
      }
      keys[g] = better < p.top_groups;                         // every element's key has been read
    }
    wave_fence();
    const float inv = 1.0f / (float)per;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LPR, W>(v, lane);
      if (e < p.E && !keys[(int)(((float)e + 0.5f) * inv)]) key[v] = 0;
    }
    wave_fence();
  }
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
    uint32_t at = ~0u;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = (uint32_t)expert_of<LPR, W>(v, lane);
      }
    const uint64_t most = lanes_reduce<LPR>(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    const uint32_t e = lanes_reduce<LPR>(best == most ? at : ~0u, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((uint32_t)expert_of<LPR, W>(v, lane) == e) key[v] = 0;
    if (lane == j % LPR) sel[j] = (int32_t)e;                  // ~0u where nothing is left
  }
  wave_fence();
}

// The same in 32 bits, where it can be shown to be the same (else false, for the whole row): k < LPR.
// Keys are a value's ordered bits with the lowest IB replaced by the expert's, counted down, so that one maximum over
// them is a value and, of equal ones, the lowest index; the next is the maximum of key - last modulo 2^32, which is
// larger for every key below the last than for any above.  k + 3 are taken, one to a lane, put in order by their
// full values (neighbours that the lost bits exchanged): the logits, a sigmoid in 64 bits, or a softmax with what it may be
// off by.  The order is certain where neighbours are further apart than that, and the last chosen than what was not
// taken could be.
//   off: a sigmoid from the hardware's exp2 and reciprocal by less than 2^-20; a softmax, whose sum of E terms adds at most
//   that many half steps along a lane and over the lanes, by less than 2^-18; the sum with the bias by half a step.
// 16-bit logits without a bias lose no bits and need no proof.  k >= LPR goes through 64 bits: 8192 x 256, k 8 and 16 (us) 5.9 and
// 15.6, with a bias 7.2 and 21.4.
// 65536 rows of 256 with a bias: 33 us, 81 us in 64 bits throughout; 2049 rows in 8 groups 12 us, 20 in 64 bits, and 23
// where one of them is not certain and both are done (1 to 9 of 16 random launches, by how far logits spread).
__device__ __forceinline__ float key_value(uint32_t key) { return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key); }
// Ordered bits of a number that is none of NaN and not -0.  Those of -inf, a masked one, and what lies below (0: not
// allowed) are at most kNone; every number's are above.
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t quick_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// The value of the lane above or below, within 16 or 64 lanes (the last one's, the first one's: some lane's).
template <int LPR>
__device__ __forceinline__ uint32_t lane_above(uint32_t v) {
  if constexpr (LPR == 16) return ror16<15>(v);
  return (uint32_t)__shfl_down((int)v, 1, 64);
}
template <int LPR>
__device__ __forceinline__ uint32_t lane_below(uint32_t v) {
  if constexpr (LPR == 16) return ror16<1>(v);
  return (uint32_t)__shfl_up((int)v, 1, 64);
}
template <int LPR>
__device__ __forceinline__ double lane_above(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)lane_above<LPR>((uint32_t)(u >> 32)) << 32 | lane_above<LPR>((uint32_t)u)));
}
template <int LPR>
__device__ __forceinline__ double lane_below(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)lane_below<LPR>((uint32_t)(u >> 32)) << 32 | lane_below<LPR>((uint32_t)u)));
}
template <int TYPE, int LPR, int J, int W>
__device__ bool select_fast(const RouteArgs& p, const float* l, const typename Logit<TYPE>::T* row, float top, float inv_sum, int lane,
                            uint32_t* keys, float* group_value, int32_t* sel) {
  constexpr int V = J * W, IB = LPR == 16 ? 8 : 10;
  constexpr uint32_t IM = (1u << IB) - 1;
  static_assert(V * LPR <= 1 << IB, "an index fits");
  const bool scored = p.bias || (p.groups > 1 && p.group_best > 1);
  const float tol = p.sigmoid ? 0x1p-20f : 0x1p-18f;
  auto score = [&](float x) {
    return p.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-x)) : __expf(x - top) * inv_sum;
  };
  uint32_t key[V];
  // NaN, which only 64 bits put in order (an infinite logit makes all of a softmax NaN), or no certainty
  bool odd = scored && !p.sigmoid && inv_sum != inv_sum;
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e0 = (j * LPR + lane) * W;
      float b[W];
      if (e0 + W <= p.E) {
        __builtin_memcpy(b, p.bias + e0, W * sizeof(float));
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) b[i] = e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float x = l[j * W + i], c = score(x) + b[i];     // a score is not -0, nor is its sum
        odd |= c != c;
        key[j * W + i] = quick_key(x == kMasked ? kMasked : c);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      odd |= l[v] != l[v];
      key[v] = quick_key(l[v] + 0.0f);                         // -0 as +0
    }
  }
  if (p.groups > 1) {
    const int per = p.E / p.groups;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LPR, W>(v, lane);
      if (e < p.E) keys[e] = p.bias || !scored ? key[v] : quick_key(l[v] == kMasked ? kMasked : score(l[v]));
    }
    wave_fence();
    for (int g = lane; g < p.groups; g += LPR) {
      uint32_t a = 0, b = 0;                                   // the two largest
      auto take = [&](uint32_t x) {
        b = max(b, min(a, x));
        a = max(a, x);
      };
      int i = 0;
      for (; i + 8 <= per; i += 8) {
        uint32_t x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = keys[g * per + i + u];
#pragma unroll
        for (int u = 0; u < 8; ++u) take(x[u]);
      }
      for (; i < per; ++i) take(keys[g * per + i]);
      const bool two = p.group_best > 1 && b > kNone;
      group_value[2 * g] = a <= kNone ? -INFINITY : two ? key_value(a) + key_value(b) : key_value(a);
      group_value[2 * g + 1] = fabsf(key_value(a)) + (two ? fabsf(key_value(b)) : 0.0f);      // what it may be off by
    }
    wave_fence();
    for (int g = lane; g < p.groups; g += LPR) {
      const float mine = group_value[2 * g], size = group_value[2 * g + 1];
      if (mine != -INFINITY && !(size < INFINITY)) odd = true;
      int better = 0, near = 0;
#pragma unroll 4
      for (int o = 0; o < p.groups; ++o) {
        const float x = group_value[2 * o], off = scored ? 4.0f * tol + 0x1p-20f * (size + group_value[2 * o + 1]) : 0.0f;
        if (o == g || x == -INFINITY) continue;
        if (x > mine + off) ++better;
        else if (x >= mine - off && (scored || o < g)) ++near; // logits are exact: an equal group of lower index is before
      }
      if (!scored) {
        better += near;
        near = 0;
      }
      if (mine != -INFINITY && better < p.top_groups && better + near >= p.top_groups) odd = true;
      keys[g] = mine != -INFINITY && better < p.top_groups;    // every element's key has been read
    }
    wave_fence();
    const float inv = 1.0f / (float)per;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<LPR, W>(v, lane);
      if (e >= p.E || !keys[(int)(((float)e + 0.5f) * inv)]) key[v] = 0;
    }
    wave_fence();
  }
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = (key[v] & ~IM) | (IM - (uint32_t)expert_of<LPR, W>(v, lane));
  const int most = min(p.k + 3, LPR);
  uint32_t last = 0, mine = 0;
  for (int j = 0; j < most; ++j) {
    uint32_t d = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) d = max(d, key[v] - last);
    d = lanes_reduce<LPR>(d, [](uint32_t a, uint32_t b) { return max(a, b); });
    const uint32_t next = last + d;
    last = next <= kNone || (j > 0 && next >= last) ? 0u : next;      // masked ones only, or nothing left
    if (lane == j) mine = last;
    if (last == 0) break;                                      // of this row: its lanes' reductions are their own
  }
  const bool live = mine != 0;
  uint32_t e = live ? IM - (mine & IM) : ~0u;
  if (TYPE == ROUTE_FP32 || p.bias) {
    double c = 0.0;
    if (live) {
      const float x = Logit<TYPE>::up(row[e]);
      c = !p.bias ? (double)x : (p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : (double)score(x)) + (double)p.bias[e];
    }
    const double off = p.bias && !p.sigmoid ? 2.0 * tol + 0x1p-21 * fabs(c) : 0.0;
    // two rounds of neighbours exchanged where the full values say so
#pragma unroll
    for (int round = 0; round < 2; ++round) {
      const bool low = ((lane + round) & 1) == 0;              // this lane and the one above, or the one below
      const uint32_t ea = lane_above<LPR>(e), eb = lane_below<LPR>(e);
      const double ca = lane_above<LPR>(c), cb = lane_below<LPR>(c);
      const uint32_t eo = low ? ea : eb;
      const double co = low ? ca : cb;
      const int other = low ? lane + 1 : lane - 1;
      if (live && other >= 0 && other < LPR && eo != ~0u) {
        const bool before = co > c || (co == c && eo < e);     // the other one is before this one
        if (before == low) {
          c = co;
          e = eo;
        }
      }
    }
    const uint32_t ea = lane_above<LPR>(e);
    const double ca = lane_above<LPR>(c);
    if (live && lane + 1 < LPR && ea != ~0u) {
      if (!(c > ca || (c == ca && e < ea))) odd = true;
      if (off > 0.0 && lane < p.k && !(c > ca + off)) odd = true;
    }
    // what was not taken is below the last key with its lost bits set, and with a bias off by what the score may be
    const double above = (double)key_value(last | IM);
    if (last != 0 && lane == p.k - 1 && !(c > above + (p.bias ? 2.0 * tol + 0x1p-21 * fabs(above) : 0.0))) odd = true;
  }
  if (lane < p.k) sel[lane] = (int32_t)e;
  wave_fence();
  return lanes_reduce<LPR>((uint32_t)odd, [](uint32_t a, uint32_t b) { return a | b; }) == 0;
}

// ----------------------------------------------------------------------------- weights
// Weights of the row's chosen experts, slot i LPR + lane, before the scale; sum over the chosen where
// they are renormalized.  The largest exponent is taken out of all of them (sigmoid(l) =
// exp(min(l, 0)) / (1 + exp(-|l|))), so that scores too small for fp32 still have their ratios.
template <int LPR, int S>
__device__ __forceinline__ void slot_weights(const RouteArgs& p, const float* l, const bool* live, float top, float inv_sum,
                                             float* w) {
  float most = kMasked;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const float x = p.sigmoid ? (l[i] > 0.0f ? 0.0f : l[i]) : l[i];
    if (live[i]) most = fmaxf(most, x);
  }
  most = lanes_max<LPR>(most);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (!p.renormalize) {
      w[i] = p.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - top) * inv_sum;
    } else if (p.sigmoid) {
      w[i] = expf((l[i] > 0.0f ? 0.0f : l[i]) - most) / (1.0f + expf(-fabsf(l[i])));
    } else {
      w[i] = expf(l[i] - most);
    }
    if (!live[i]) w[i] = 0.0f;
    sum += w[i];
  }
  if (!p.renormalize) return;
  sum = lanes_sum<LPR>(sum);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < S; ++i) w[i] = sum == w[i] ? live[i] : w[i] * inv;      // one expert alone: 1
}
// The largest logit of the row (0 without one) and 1 / sum of exp(l - top), of a softmax over all experts.
template <int LPR, int V>
__device__ __forceinline__ float row_top(const float* l) {
  float top = kMasked;
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, l[v]);
  top = lanes_max<LPR>(top);
  return top == kMasked ? 0.0f : top;
}
template <int LPR, int V>
__device__ __forceinline__ float row_inv_sum(const float* l, float top) {
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += expf(l[v] - top);
  sum = lanes_sum<LPR>(sum);
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

// ----------------------------------------------------------------------------- kernels
template <int TYPE, int LPR, int J>
__global__ __launch_bounds__(RT) void route_kernel(RouteArgs p) {
  using L = Logit<TYPE>;
  constexpr int W = L::W, V = J * W, ROWS = RT / LPR;
  extern __shared__ uint64_t s_keys[];                         // [ROWS][E] where there are groups
  __shared__ uint64_t s_group[ROWS][kRouteMaxGroups];
  __shared__ int32_t s_sel[ROWS][kRouteMaxK];
  const int lane = threadIdx.x % LPR, r = threadIdx.x / LPR;
  const int64_t t = ((int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks) * ROWS + r;
  const bool in = t < p.T;                                     // the other rows run along, as rows of nothing
  const typename L::T* row = static_cast<const typename L::T*>(p.logits) + (in ? t : 0) * p.ld;
  float l[V];
  load_row<TYPE, LPR, J>(row, in ? p.E : 0, lane, l);
  const float top = p.sigmoid ? 0.0f : row_top<LPR, V>(l);
  const bool sums = !p.sigmoid && (!p.renormalize || p.bias || (p.groups > 1 && p.group_best > 1));
  const float inv_sum = sums ? row_inv_sum<LPR, V>(l, top) : 0.0f;
  // the wave's rows together, so that all its lanes are there
  const bool fast = p.k < LPR && select_fast<TYPE, LPR, J, W>(p, l, row, top, inv_sum, lane, reinterpret_cast<uint32_t*>(s_keys + (int64_t)r * p.E),
                                                              reinterpret_cast<float*>(s_group[r]), s_sel[r]);
  if (!__all(fast)) select_exact<LPR, J, W>(p, l, top, lane, s_keys + (int64_t)r * p.E, s_group[r], s_sel[r]);
  auto finish = [&](auto slots) {
    constexpr int S = decltype(slots)::value;
    int32_t e[S];
    float x[S], w[S];
    bool live[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int j = i * LPR + lane;
      e[i] = j < p.k ? s_sel[r][j] : -1;
      live[i] = e[i] >= 0;
      x[i] = live[i] ? L::up(row[e[i]]) : 0.0f;
    }
    slot_weights<LPR, S>(p, x, live, top, inv_sum, w);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int j = i * LPR + lane;
      if (in && j < p.k) {
        p.experts[t * p.k + j] = e[i];
        p.probs[t * p.k + j] = live[i] ? w[i] * p.scale : 0.0f;
      }
    }
  };
  if (p.k <= LPR) finish(std::integral_constant<int, 1>{});
  else finish(std::integral_constant<int, kRouteMaxK / LPR>{});
}

// dlogits of a row, all of it: with g_j = scale dprobs_j and w_j the weights before the scale
//   softmax                 p_e (sum of g_j at e - sum_j g_j w_j)
//   softmax, renormalized   w_j (g_j - sum g w) at the chosen, 0 elsewhere
//   sigmoid                 g_j s_j (1 - s_j) at the chosen
//   sigmoid, renormalized   w_j (g_j - sum g w) (1 - s_j) at the chosen
// The slots' parts are added to the row in LDS one slot after the other, so that an expert named twice has the
// sum, in a fixed order.
template <int TYPE, int LPR, int J>
__global__ __launch_bounds__(RT) void route_backward_kernel(RouteArgs p) {
  using L = Logit<TYPE>;
  constexpr int W = L::W, V = J * W, ROWS = RT / LPR, S = kRouteMaxK / LPR;
  __shared__ float s_row[ROWS][V * LPR];
  const int lane = threadIdx.x % LPR, r = threadIdx.x / LPR;
  const int64_t t = ((int64_t)blockIdx.x + (int64_t)blockIdx.y * p.row_blocks) * ROWS + r;
  const bool in = t < p.T;
  const typename L::T* row = static_cast<const typename L::T*>(p.logits) + (in ? t : 0) * p.ld;
  const bool dense = !p.sigmoid && !p.renormalize;
  float l[V];
  float top = 0.0f, inv_sum = 0.0f;
  if (dense) {
    load_row<TYPE, LPR, J>(row, in ? p.E : 0, lane, l);
    top = row_top<LPR, V>(l);
    inv_sum = row_inv_sum<LPR, V>(l, top);
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) s_row[r][(j * LPR + lane) * W + i] = 0.0f;
  int32_t e[S];
  float x[S], w[S], g[S];
  bool live[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int j = i * LPR + lane;
    e[i] = in && j < p.k ? p.experts[t * p.k + j] : -1;
    live[i] = (uint32_t)e[i] < (uint32_t)p.E;
    x[i] = live[i] ? L::up(row[e[i]]) : 0.0f;
    live[i] = live[i] && x[i] != kMasked;
    g[i] = live[i] ? p.scale * p.dprobs[t * p.k + j] : 0.0f;
  }
  slot_weights<LPR, S>(p, x, live, top, inv_sum, w);
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < S; ++i) dot += live[i] ? g[i] * w[i] : 0.0f;
  dot = lanes_sum<LPR>(dot);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (p.renormalize) g[i] = w[i] * (g[i] - dot);
    else if (p.sigmoid) g[i] = g[i] * w[i];
    if (p.sigmoid) g[i] = g[i] / (1.0f + expf(x[i]));
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < S; ++i)
    for (int j = 0; j < LPR && i * LPR + j < p.k; ++j) {
      if (lane == j && live[i]) s_row[r][e[i]] += g[i];
      wave_fence();
    }
  if (!in) return;
  typename L::T* out = static_cast<typename L::T*>(p.dlogits) + t * p.ld_dlogits;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e0 = (j * LPR + lane) * W;
    if (e0 >= p.E) continue;
    typename L::T y[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float d = s_row[r][e0 + i];
      if (dense) d = l[j * W + i] == kMasked ? 0.0f : expf(l[j * W + i] - top) * inv_sum * (d - dot);
      y[i] = L::down(d);
    }
    if (e0 + W <= p.E) {
      __builtin_memcpy(out + e0, y, 16);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (e0 + i < p.E) out[e0 + i] = y[i];
    }
  }
}

// ----------------------------------------------------------------------------- launches
template <int TYPE, int LPR, int J>
static hipError_t run_route(RouteArgs p, bool backward, hipStream_t s) {
  constexpr int ROWS = RT / LPR;
  const FoldedGrid g = fold_grid((p.T + ROWS - 1) / ROWS, RT);
  p.row_blocks = g.x;
  if (backward)
    hipLaunchKernelGGL((route_backward_kernel<TYPE, LPR, J>), dim3(g.x, g.y), dim3(RT), 0, s, p);
  else
    hipLaunchKernelGGL((route_kernel<TYPE, LPR, J>), dim3(g.x, g.y), dim3(RT), p.groups > 1 ? sizeof(uint64_t) * ROWS * p.E : 0, s, p);
  return hipGetLastError();
}
// The fewest lanes and loads that hold the row.
template <int TYPE>
static hipError_t run_route(const RouteArgs& p, bool backward, hipStream_t s) {
  constexpr int W = Logit<TYPE>::W;
  if (p.E <= 16 * W) return run_route<TYPE, 16, 1>(p, backward, s);
  if (p.E <= 32 * W) return run_route<TYPE, 16, 2>(p, backward, s);
  if constexpr (W == 4) {
    if (p.E <= 64 * W) return run_route<TYPE, 16, 4>(p, backward, s);
    if (p.E <= 128 * W) return run_route<TYPE, 64, 2>(p, backward, s);
    return run_route<TYPE, 64, 4>(p, backward, s);
  } else {
    if (p.E <= 64 * W) return run_route<TYPE, 64, 1>(p, backward, s);
    return run_route<TYPE, 64, 2>(p, backward, s);
  }
}
static hipError_t run_route(const RouteArgs& p, bool backward, hipStream_t s) {
  if (p.type == ROUTE_BF16) return run_route<ROUTE_BF16>(p, backward, s);
  if (p.type == ROUTE_FP16) return run_route<ROUTE_FP16>(p, backward, s);
  return run_route<ROUTE_FP32>(p, backward, s);
}
hipError_t launch_route(const RouteArgs& p, hipStream_t s) { return run_route(p, false, s); }
hipError_t launch_route_backward(const RouteArgs& p, hipStream_t s) { return run_route(p, true, s); }

}  // namespace gmlp
