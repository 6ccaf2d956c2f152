// route_experts.cuh -- the router of an expert layer: scores of the experts from
// their logits, the best experts of each row with their weights, and the
// gradient of the logits.
//
//   s_e = 1 / (1 + exp(-l_e))   or   exp(l_e) / sum exp(l)
//   key_e = s_e + bias_e                       (the bias chooses, it does not weigh)
//   of `groups` equal groups of experts those with the largest sums of their
//   `group_best` best keys are kept; of their experts the `top` largest keys
//   w_e = scale * s_e, or scale * s_e / (sum of the chosen s)
//
// The choice is the one that exact arithmetic makes (ties: the lowest index),
// which 32 bits cannot always tell. Where no bias takes part and groups go by
// their best expert, experts are compared by their logits, which order them as
// their scores do. Otherwise keys are computed in 32 bits with a known error, and
// a row where two keys that decide lie closer than that goes through
// route_careful(), in 64 bits. Two experts of the same logit and the same bias
// are a tie and decided as such: with 16-bit logits and biases that move in
// steps, that is the common case.
//
// A row is the work of LANES lanes of a warp, each with up to PER neighbouring
// experts in registers (a group's experts in lanes of their own). A lane's key is
// one 32-bit integer: the key as an integer of the same order, its lowest bits
// replaced by the expert's place in the lane, so that one maximum over the lane
// and one over the lanes give the next pick and where it came from.
#pragma once

#include <cfloat>
#include <cstdint>

#include "common.cuh"

namespace sptg {

enum RouteType : int { ROUTE_F16 = 0, ROUTE_BF16 = 1, ROUTE_F32 = 2 };

constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_TOP = 16;
constexpr int ROUTE_MAX_GROUPS = 32;
constexpr int ROUTE_WARPS = 4;  // of a block

struct RouteParams {
  const void* logits;
  int64_t ld, rows;      // elements between rows
  const float* bias;     // or null
  float* weights;        // rows x top
  int32_t* experts;      // rows x top
  int E, top, sigmoid, renorm;
  float scale;
  int groups, top_groups, group_best;
  int size;              // experts of a group
  int lanes_log2;        // lanes of a group
  int chunk;             // experts of a lane
  int wide, wide_bias;   // 16-byte loads of logits and bias
};

struct RouteGradParams {
  const void* logits;
  int64_t ld, rows;
  const int32_t* experts;  // rows x top
  const float* dweights;   // rows x top
  void* dlogits;
  int64_t ldd;
  int E, top, sigmoid, renorm;
  float scale;
  int wide;
};

template <int TYPE>
__device__ __forceinline__ float route_load(const void* p, int64_t i) {
  if constexpr (TYPE == ROUTE_F32)
    return static_cast<const float*>(p)[i];
  else if constexpr (TYPE == ROUTE_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else
    return __half2float(static_cast<const __half*>(p)[i]);
}

// 16 bytes of logits, 4 or 8 of them.
template <int TYPE>
__device__ __forceinline__ void route_unpack(const uint4& v, float* l) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == ROUTE_F32) {
      l[i] = __uint_as_float(w[i]);
    } else if constexpr (TYPE == ROUTE_BF16) {
      l[2 * i] = __uint_as_float(w[i] << 16);
      l[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      l[2 * i] = f.x;
      l[2 * i + 1] = f.y;
    }
  }
}

// A float as an unsigned integer of the same order (-0 as +0), and back.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A logistic function whose small values keep their relative precision.
__device__ __forceinline__ float logistic(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

template <int LANES>
__device__ __forceinline__ float route_sum(float v, uint32_t mask) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}

// The choice of one row in 64 bits, by the row's lanes: this lane's pick (lane i
// has the i-th), or -1. Called for rows that 32 bits do not settle, a few in a
// thousand: it reads its inputs anew and holds nothing in the fast path's registers.
template <int TYPE, int LANES, int PER>
__device__ __noinline__ int route_careful(const RouteParams& p, int64_t row, int first, int count,
                                          bool direct, uint32_t mask) {
  const int sub = static_cast<int>(lane_id()) & (LANES - 1);
  const int g = sub >> p.lanes_log2;
  const auto sum = [&](double v) {
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
  };
  const auto largest = [&](double v) {
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(mask, v, o));
    return v;
  };
  double key[PER];
  double m = -INFINITY;
  for (int j = 0; j < PER; ++j) {
    key[j] = j < count ? route_load<TYPE>(p.logits, row * p.ld + first + j) : -INFINITY;
    m = fmax(m, key[j]);
  }
  m = largest(m);
  double z = 1.0;
  if (!p.sigmoid) {
    z = 0.0;
    for (int j = 0; j < PER; ++j)
      if (key[j] > -INFINITY) z += exp(key[j] - m);
    z = sum(z);
  }
  for (int j = 0; j < PER; ++j) {
    if (!(key[j] > -INFINITY)) continue;
    const double b = p.bias ? static_cast<double>(p.bias[first + j]) : 0.0;
    if (!direct)  // (else logits are compared, here as there)
      key[j] = p.sigmoid ? 1.0 / (1.0 + exp(-key[j])) : exp(key[j] - m) / z;
    key[j] = direct && b > -INFINITY ? key[j] : key[j] + b;
  }
  if (p.groups > 1) {
    double t1 = -INFINITY, t2 = -INFINITY;
    for (int j = 0; j < PER; ++j) {
      t2 = fmax(t2, fmin(t1, key[j]));
      t1 = fmax(t1, key[j]);
    }
    for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
      const double a1 = __shfl_xor_sync(mask, t1, o), a2 = __shfl_xor_sync(mask, t2, o);
      t2 = fmax(fmin(t1, a1), fmax(t2, a2));
      t1 = fmax(t1, a1);
    }
    const double score = p.group_best == 2 && t2 > -INFINITY ? t1 + t2 : t1;
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const double other = __shfl_sync(mask, score, o << p.lanes_log2, LANES);
      rank += other > score || (other == score && o < g);
    }
    if (rank >= p.top_groups)
      for (int j = 0; j < PER; ++j) key[j] = -INFINITY;
  }
  int mine = -1;
  for (int i = 0; i < p.top; ++i) {
    double best = -INFINITY;
    int at = INT32_MAX;
    for (int j = 0; j < PER; ++j)
      if (key[j] > best) {
        best = key[j];
        at = first + j;
      }
    for (int o = LANES / 2; o > 0; o >>= 1) {
      const double b = __shfl_xor_sync(mask, best, o);
      const int a = __shfl_xor_sync(mask, at, o);
      if (b > best || (b == best && a < at)) {
        best = b;
        at = a;
      }
    }
    if (sub == i && at != INT32_MAX) mine = at;
    for (int j = 0; j < PER; ++j)
      if (first + j == at) key[j] = -INFINITY;
  }
  return mine;
}

template <int TYPE, int LANES, int PER>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    route_experts_kernel(const __grid_constant__ RouteParams p) {
  constexpr int N = TYPE == ROUTE_F32 ? 4 : 8;  // logits in 16 bytes
  constexpr uint32_t PLACE = PER - 1;           // a key's lowest bits: PER - 1 - place in the lane
  // What separates two keys for certain, relative to their size: the roundings of
  // two scores (expf, the division, the sum over the experts: 2^-20 each) and the
  // bits that the place takes (2^-20 with 8 experts a lane), twice over.
  constexpr float APART = PER / 8 * 3.814697265625e-06f;  // 2^-18
  const int lane = threadIdx.x & 31, sub = lane & (LANES - 1);
  const uint32_t mask = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (lane - sub);
  const int64_t at =
      (static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5)) * (32 / LANES) + lane / LANES;
  const int64_t row = min(at, p.rows - 1);  // (lanes past the end repeat the last row and store nothing)
  const int g = sub >> p.lanes_log2, q = sub & ((1 << p.lanes_log2) - 1);
  const int first = g * p.size + q * p.chunk;
  const int count = g < p.groups ? max(0, min(p.chunk, p.size - q * p.chunk)) : 0;
  grid_dependency_wait();
  float l[PER];
  if (p.wide) {
    const uint4* src =
        reinterpret_cast<const uint4*>(static_cast<const char*>(p.logits) + (row * p.ld + first) * (16 / N));
#pragma unroll
    for (int k = 0; k < PER / N; ++k) {
      if (k * N < count) {
        route_unpack<TYPE>(src[k], &l[k * N]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) l[k * N + j] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      l[j] = j < count ? route_load<TYPE>(p.logits, row * p.ld + first + j) : -INFINITY;
  }
  grid_launch_dependents();
  bool bad = false;
  uint32_t top_l = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    bad = bad || l[j] != l[j];
    top_l = max(top_l, order_bits(l[j]));
  }
  const float m = from_order_bits(__reduce_max_sync(mask, top_l));
  bad = bad || (!p.sigmoid && m == INFINITY);
  float z = 1.0f;  // what a softmax divides by, where it counts
  if (!p.sigmoid && (!p.renorm || p.bias != nullptr || (p.groups > 1 && p.group_best == 2))) {
    z = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) z += l[j] > -INFINITY ? expf(l[j] - m) : 0.0f;
    z = route_sum<LANES>(z, mask);
  }
  const float rz = 1.0f / z;
  uint32_t k[PER];
  float b_most = 0.0f;  // the largest bias by magnitude, of experts that can be chosen
  float b[PER];
  if (p.bias != nullptr) {
    if (p.wide_bias) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        const float4 v = 4 * i < count ? *reinterpret_cast<const float4*>(p.bias + first + 4 * i)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        b[4 * i] = v.x;
        b[4 * i + 1] = v.y;
        b[4 * i + 2] = v.z;
        b[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) b[j] = j < count ? p.bias[first + j] : 0.0f;
    }
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (b[j] == -INFINITY) {
        l[j] = -INFINITY;  // (the softmax has it still)
        b[j] = 0.0f;
      }
      most = max(most, __float_as_uint(b[j]) & 0x7fffffffu);
    }
    b_most = __uint_as_float(__reduce_max_sync(mask, most));
    bad = bad || b_most != b_most;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) b[j] = 0.0f;
  }
  const bool biased = b_most != 0.0f;
  // Whether logits stand for the keys: exactly, if they have 16 bits.
  const bool direct = !biased && (p.groups == 1 || p.group_best == 1);
  const bool exact = direct && TYPE != ROUTE_F32;
  // How far keys are apart for certain, relative to their size. A softmax's
  // exponent is rounded in proportion to its distance from the largest.
  float apart_rel = APART;
  if (!direct && !p.sigmoid) {
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < PER; ++j) least = l[j] > -INFINITY ? min(least, order_bits(l[j])) : least;
    least = __reduce_min_sync(mask, least);
    if (least != 0xffffffffu) apart_rel *= 1.0f + (m - from_order_bits(least)) * 0.0625f;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    float key = l[j];
    if (!direct) key = (p.sigmoid ? logistic(l[j]) : expf(l[j] - m) * rz) + b[j];
    k[j] = l[j] > -INFINITY ? (order_bits(key) & ~PLACE) | (PLACE - j) : 0u;
  }
  bool unsettled = false;
  if (p.groups > 1) {
    uint32_t t1 = 0, t2 = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      t2 = max(t2, min(t1, k[j]));
      t1 = max(t1, k[j]);
    }
    for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
      const uint32_t a1 = __shfl_xor_sync(mask, t1, o), a2 = __shfl_xor_sync(mask, t2, o);
      t2 = max(min(t1, a1), max(t2, a2));
      t1 = max(t1, a1);
    }
    uint32_t score = t1 & ~PLACE;
    if (p.group_best == 2 && t2 != 0)
      score = order_bits(from_order_bits(t1 & ~PLACE) + from_order_bits(t2 & ~PLACE));
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const uint32_t other = __shfl_sync(mask, score, o << p.lanes_log2, LANES);
      rank += other > score || (other == score && o < g);
    }
    const bool kept = rank < p.top_groups;
    if (!exact) {
      const uint32_t worst = __reduce_min_sync(mask, kept ? score : 0xffffffffu);
      const uint32_t next = __reduce_max_sync(mask, kept ? 0u : score);
      const float w = from_order_bits(worst);
      unsettled = next != 0 && !(w - from_order_bits(next) > 2.0f * apart_rel * (fabsf(w) + 4.0f * b_most));
    }
    if (!kept) {
#pragma unroll
      for (int j = 0; j < PER; ++j) k[j] = 0;
    }
  }
  // The picks: lane i keeps the i-th key and the lane that it came from.
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) best = max(best, k[j]);
  uint32_t my_key = 0;
  int my_lane = 0;
  for (int i = 0; i < p.top; ++i) {
    const uint32_t most = __reduce_max_sync(mask, best & ~PLACE);
    const int from = __ffs(__ballot_sync(mask, (best & ~PLACE) == most)) - 1;  // (the lowest of a tie)
    const uint32_t key = __shfl_sync(mask, best, from);
    if (sub == i) {
      my_key = key;
      my_lane = from;
    }
    if (lane == from) {
      best = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        k[j] = k[j] == key ? 0u : k[j];
        best = max(best, k[j]);
      }
    }
  }
  const bool chosen = sub < p.top;
  int pick = -1;
  if (chosen && my_key != 0) {
    const int s = my_lane & (LANES - 1);
    pick = (s >> p.lanes_log2) * p.size + (s & ((1 << p.lanes_log2) - 1)) * p.chunk +
           static_cast<int>(PLACE - (my_key & PLACE));
  }
  float my_l = pick >= 0 ? route_load<TYPE>(p.logits, row * p.ld + pick) : -INFINITY;
  if (!exact) {
    const float my_b = pick >= 0 && p.bias ? p.bias[pick] : 0.0f;
    const float key = from_order_bits(my_key & ~PLACE);
    const float apart = direct ? 0.0f : apart_rel * (fabsf(key) + b_most);
    // two picks in doubt, unless they are a tie (logits: unless in order)
    const uint32_t n_key = __shfl_down_sync(mask, my_key, 1, LANES);
    const int n_pick = __shfl_down_sync(mask, pick, 1, LANES);
    const float n_l = __shfl_down_sync(mask, my_l, 1, LANES);
    const float n_b = __shfl_down_sync(mask, my_b, 1, LANES);
    if (sub + 1 < p.top && n_key != 0 && !(key - from_order_bits(n_key & ~PLACE) > apart)) {
      const bool tie = my_l == n_l && my_b == n_b && pick < n_pick;
      unsettled = unsettled || !(tie || (direct && my_l > n_l));
    }
    // the last pick and those that were not picked
    const int last = (lane - sub) + p.top - 1;
    const uint32_t last_key = __shfl_sync(mask, my_key, last);
    const float last_l = __shfl_sync(mask, my_l, last), last_b = __shfl_sync(mask, my_b, last);
    const float last_apart = __shfl_sync(mask, apart, last);
    const float last_f = from_order_bits(last_key & ~PLACE);
    if (last_key != 0 && best != 0 && !(last_f - from_order_bits(best & ~PLACE) > last_apart)) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (k[j] != 0 && !(last_f - from_order_bits(k[j] & ~PLACE) > last_apart))
          unsettled = unsettled || !(l[j] == last_l && b[j] == last_b);
    }
    if (__ballot_sync(mask, unsettled) != 0 && __ballot_sync(mask, bad) == 0) {
      pick = route_careful<TYPE, LANES, PER>(p, row, first, count, direct, mask);
      my_l = pick >= 0 ? route_load<TYPE>(p.logits, row * p.ld + pick) : -INFINITY;
    }
  }
  // The weights. Renormalised ones relative to the largest chosen score, so that
  // scores that all lie near zero keep their ratios.
  float w;
  if (p.renorm) {
    const uint32_t ml = __reduce_max_sync(mask, pick >= 0 ? order_bits(my_l) : 0u);
    const float ref = from_order_bits(ml);
    if (p.sigmoid) {
      const float d = (fminf(my_l, 0.0f) - fminf(ref, 0.0f)) -
                      (log1pf(expf(-fabsf(my_l))) - log1pf(expf(-fabsf(ref))));
      w = pick >= 0 ? expf(d) : 0.0f;
    } else {
      w = pick >= 0 ? expf(my_l - ref) : 0.0f;
    }
    const float total = route_sum<LANES>(w, mask);
    w = pick >= 0 ? w / total : 0.0f;
  } else {
    w = pick < 0 ? 0.0f : p.sigmoid ? logistic(my_l) : expf(my_l - m) * rz;
  }
  w *= p.scale;
  if (__ballot_sync(mask, bad) != 0) {  // a NaN in the row (or +inf under a softmax)
    pick = sub;
    w = NAN;
  }
  if (chosen && at < p.rows) {
    p.weights[at * p.top + sub] = w;
    p.experts[at * p.top + sub] = pick;
  }
}

// Gradient of the logits, a warp to a row. With c the chosen experts, g the
// weights' gradient times scale:
//
//   sigmoid               d_c = g_c s_c (1 - s_c)
//   sigmoid, renormalised d_c = (g_c - sum g u) u_c (1 - s_c)      u: renormalised scores
//   softmax, renormalised d_c = (g_c - sum g u) u_c
//   softmax               d_e = s_e ([e chosen] g_e - sum g s)      for every expert
//
// Only the last reads all logits. The row is written first (zeros, or -s sum g s),
// then the chosen experts' values over it.
template <int TYPE>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    route_experts_dlogits_kernel(const __grid_constant__ RouteGradParams p) {
  constexpr int N = TYPE == ROUTE_F32 ? 4 : 8;
  constexpr int OUT = TYPE == ROUTE_F32 ? OUT_F32 : TYPE == ROUTE_BF16 ? OUT_BF16 : OUT_F16;
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (row >= p.rows) return;
  int e = -1;
  float g = 0.0f, l = -INFINITY;
  if (lane < p.top) {
    e = p.experts[row * p.top + lane];
    if (e < 0 || e >= p.E) e = -1;
    if (e >= 0) {
      g = p.dweights[row * p.top + lane] * p.scale;
      l = route_load<TYPE>(p.logits, row * p.ld + e);
    }
  }
  const bool full = !p.sigmoid && !p.renorm;
  const char* src = static_cast<const char*>(p.logits) + row * p.ld * (16 / N);
  char* dst = static_cast<char*>(p.dlogits) + row * p.ldd * (16 / N);
  float m = -INFINITY, rz = 0.0f;
  if (full) {
    float z = 0.0f;
    if (p.wide) {
      for (int i = lane; i < p.E / N; i += 32) {
        float v[N];
        route_unpack<TYPE>(reinterpret_cast<const uint4*>(src)[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
      }
    } else {
      for (int i = lane; i < p.E; i += 32) m = fmaxf(m, route_load<TYPE>(src, i));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(ALL, m, o));
    if (p.wide) {
      for (int i = lane; i < p.E / N; i += 32) {
        float v[N];
        route_unpack<TYPE>(reinterpret_cast<const uint4*>(src)[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) z += v[j] == -INFINITY ? 0.0f : expf(v[j] - m);
      }
    } else {
      for (int i = lane; i < p.E; i += 32) {
        const float v = route_load<TYPE>(src, i);
        z += v == -INFINITY ? 0.0f : expf(v - m);
      }
    }
    rz = 1.0f / route_sum<32>(z, ALL);
  }
  // scores of the chosen (u: those that the weights are) and the sum of g u
  float s = 0.0f, u;
  if (p.renorm) {
    const float ref = from_order_bits(__reduce_max_sync(ALL, e >= 0 ? order_bits(l) : 0u));
    float x = l - ref;
    if (p.sigmoid) {
      s = logistic(l);
      x = (fminf(l, 0.0f) - fminf(ref, 0.0f)) - (log1pf(expf(-fabsf(l))) - log1pf(expf(-fabsf(ref))));
    }
    u = e >= 0 ? expf(x) : 0.0f;
    const float total = route_sum<32>(u, ALL);
    u = e >= 0 ? u / total : 0.0f;
  } else {
    u = e < 0 ? 0.0f : p.sigmoid ? logistic(l) : l == -INFINITY ? 0.0f : expf(l - m) * rz;
    s = u;
  }
  const float dot = p.sigmoid && !p.renorm ? 0.0f : route_sum<32>(g * u, ALL);
  // an expert named twice gets both gradients (its score stands twice in the sums)
  float own = 0.0f;
  for (int i = 0; i < p.top; ++i) {
    const int oe = __shfl_sync(ALL, e, i);
    const float og = __shfl_sync(ALL, g, i);
    if (oe == e) own += p.renorm ? og - dot : og;
  }
  float d = own * u;
  if (full) d = u * (own - dot);
  // 1 - s, without cancellation
  if (p.sigmoid) d *= logistic(-l);
  const float back = full ? -dot : 0.0f;
  if (p.wide) {
    for (int i = lane; i < p.E / N; i += 32) {
      float v[N];
      if (full) {
        route_unpack<TYPE>(reinterpret_cast<const uint4*>(src)[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] == -INFINITY ? 0.0f : expf(v[j] - m) * rz * back;
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 0.0f;
      }
      store_row_group<OUT>(dst, i * N, v, N);
    }
  } else {
    for (int i = lane; i < p.E; i += 32) {
      float v = 0.0f;
      if (full) {
        v = route_load<TYPE>(src, i);
        v = v == -INFINITY ? 0.0f : expf(v - m) * rz * back;
      }
      store_out<OUT>(dst, i, v);
    }
  }
  __syncwarp();  // (orders the row's stores before those of the chosen)
  if (e >= 0) store_out<OUT>(dst, e, d);
  grid_launch_dependents();
}

}  // namespace sptg
