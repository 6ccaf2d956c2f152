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
// their scores do. Otherwise keys are computed in 32 bits with a known error, and what
// decides where two lie closer than that is:
// - without a bias, logits for experts, and for sums of two scores their difference, formed so
//   that scores of any size count (route_by_logits);
// - with a bias, the keys in 44 bits (Pair), and if that does not settle it, in 64
//   (route_careful). Keys, or sums of two, that differ by less than 2^-42 of their size and the
//   largest bias's may count as equal.
// Two experts of the same logit and the same bias are a tie and decided as such: with 16-bit
// logits and biases that move in steps, that is the common case. (Without a bias rows in
// doubt wait until all registers are free: 32768 rows of 256 bf16 logits in 8 groups take 41 us,
// and 145 us where most scores lie within 2^-20 of 1; settled on the spot 44 and 950 us, and
// rows of 64 experts, which never are in doubt, 10.3 instead of 8.8 us.)
//
// A row is the work of LANES lanes of a warp, each with up to PER neighbouring
// experts in registers (a group's experts in lanes of their own). A lane's key is
// one 32-bit integer: the key as an integer of the same order, its lowest bits
// replaced by the expert's place in the lane. A lane sorts its keys (a comparison
// is a minimum and a maximum), so the next pick is the largest of the lanes' first
// keys, and the two best of a group are at hand.
//
// Bound by the issue of instructions (32768 rows of 256 f32 logits, bias, 8 groups, 8 picks:
// 36 us, of which memory needs 5; two thirds of the issue slots are taken), so whatever one row needs in a few lanes
// only is done for several at once: a warp makes the choices of up to 4 rows first
// (8 places each; with more than 8 picks 2 of 16), then looks for doubts and
// works out the weights of all of them, one place to a lane.
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
  int slots_log2;        // lanes of a row's picks: 8 or 16
  int turns;             // of 32 / LANES rows that a warp takes
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

// A float (not -0) as an unsigned integer of the same order, and back.
__device__ __forceinline__ uint32_t order_bits(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// 1 / (1 + exp(-l)) for the comparison of keys, in four instructions: off by 2^-21 and
// by l times 2^-24 of itself.
__device__ __forceinline__ float logistic_key(float l) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

// A logistic function whose small values keep their relative precision.
__device__ __forceinline__ float logistic(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// The largest of three, NaN if any is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// Sums and maxima of LANES neighbouring lanes; all of a warp take part, or those of the mask. (Reductions
// and votes with a mask of their own for each part of a warp run part by part: 32768
// rows of 128 experts, two to a warp, 23 us.)
template <int LANES>
__device__ __forceinline__ float route_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t route_max(uint32_t v, uint32_t mask = 0xffffffffu) {
  if constexpr (LANES == 32) return __reduce_max_sync(0xffffffffu, v);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(mask, v, o));
  return v;
}

// Keys in falling order, by a network of comparisons: halves sorted, then merged
// (Batcher's odd-even merge of every R-th key from LO on).
template <int LO, int LEN, int R, int N>
__device__ __forceinline__ void merge_down(uint32_t (&k)[N]) {
  const auto exchange = [&](int a, int b) {
    const uint32_t hi = max(k[a], k[b]);
    k[b] = min(k[a], k[b]);
    k[a] = hi;
  };
  if constexpr (2 * R < LEN) {
    merge_down<LO, LEN, 2 * R>(k);
    merge_down<LO + R, LEN, 2 * R>(k);
#pragma unroll
    for (int i = LO + R; i + R < LO + LEN; i += 2 * R) exchange(i, i + R);
  } else {
    exchange(LO, LO + R);
  }
}
template <int LO, int LEN, int N>
__device__ __forceinline__ void sort_down(uint32_t (&k)[N]) {
  if constexpr (LEN > 1) {
    sort_down<LO, LEN / 2>(k);
    sort_down<LO + LEN / 2, LEN / 2>(k);
    merge_down<LO, LEN, 1>(k);
  }
}

// What separates two keys for certain. A key is a score and a bias of at most
// b_most, s its size with the bias's: relative to s the score is off by 2^-21 and
// by its logit's (or its distance from the largest logit) times 2^-23, which is
// no more than -log2(s) where that counts; the place's bits take 2^-20 (8 experts
// a lane). A softmax's sum adds 2^-20. (Below 2^-100 nothing is certain: scores that
// small lose bits.)
template <int PER>
__device__ __forceinline__ float route_apart(float key, float b_most, bool sigmoid) {
  const float APART = PER / 8 * (sigmoid ? 1.9073486e-06f : 3.814697265625e-06f);  // 2^-19, 2^-18
  const float s = fabsf(key) + b_most;
  return s > 0x1p-100f ? APART * s * (1.0f + 0.0625f * fmaxf(0.0f, -__log2f(s))) : INFINITY;
}

// Numbers as unevaluated sums of two floats, with error-free sums and products
// (Dekker, Knuth): 2^-44 relative. Keys are compared in them where floats do not
// settle a choice; on this GPU a double's exponential and division take three
// times as long, and with thousands of rows there always is one in doubt that the
// others wait for.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair pair_norm(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair pair_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = pair_sum(a.hi, b.hi), t = pair_sum(a.lo, b.lo);
  const Pair u = pair_norm(s.hi, __fadd_rn(s.lo, t.hi));
  return pair_norm(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.hi, b.hi), e = __fmaf_rn(a.hi, b.hi, -p);
  return pair_norm(p, __fadd_rn(e, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
__device__ __forceinline__ Pair over(Pair a, Pair b) {
  float c;  // about 1 / b
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(b.hi));
  const float q = __fmul_rn(a.hi, c);
  const Pair qb = Pair{q, 0.0f} * b;
  const float r = __fadd_rn(__fsub_rn(__fsub_rn(a.hi, qb.hi), qb.lo), a.lo);
  return pair_norm(q, __fmul_rn(r, c));
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ bool operator==(Pair a, Pair b) { return a.hi == b.hi && a.lo == b.lo; }
// exp(x) for x <= 0 (values below 2^-126 lose their precision): x = n ln 2 + r, the
// power series of exp(r), |r| <= 0.35: terms from r^7 / 7! on, below 2^-22, in one float.
__device__ __forceinline__ Pair pair_exp(Pair x) {
  if (!(x.hi > -104.0f)) return {0.0f, 0.0f};
  const float n = rintf(x.hi * 1.44269504f);
  // ln 2 = 0x1.63p-1 (so that n times it is exact) - 0x1.bd0106p-13 + c
  const float c = 0x1.cf79acp-40f;  // ln 2 - 0x1.63p-1 + 0x1.bd0106p-13
  const float t = __fmaf_rn(-n, 0x1.63p-1f, x.hi);
  const float m = __fmul_rn(n, 0x1.bd0106p-13f), me = __fmaf_rn(n, 0x1.bd0106p-13f, -m);
  Pair r = pair_sum(t, m);
  r = pair_norm(r.hi, __fadd_rn(r.lo, __fadd_rn(__fadd_rn(me, x.lo), __fmul_rn(-n, c))));
  // 1/7! ... 1/12!
  float f = 2.0876757e-9f;
  f = __fmaf_rn(f, r.hi, 2.5052108e-8f);
  f = __fmaf_rn(f, r.hi, 2.7557319e-7f);
  f = __fmaf_rn(f, r.hi, 2.7557319e-6f);
  f = __fmaf_rn(f, r.hi, 2.4801587e-5f);
  f = __fmaf_rn(f, r.hi, 1.9841270e-4f);
  Pair v = {__fmul_rn(f, r.hi), 0.0f};
  v = v + Pair{1.38888892e-3f, -3.3631094e-11f};  // 1/6!
  v = v * r + Pair{8.33333377e-3f, -4.3461720e-10f};
  v = v * r + Pair{4.16666679e-2f, -1.2417635e-9f};
  v = v * r + Pair{1.66666672e-1f, -4.9670538e-9f};
  v = v * r + Pair{0.5f, 0.0f};
  v = v * r + Pair{1.0f, 0.0f};
  v = v * r + Pair{1.0f, 0.0f};
  const float scale = ldexpf(1.0f, static_cast<int>(n));
  return {v.hi * scale, v.lo * scale};
}

// The score with its bias. z: the softmax's sum, of exponentials from the largest logit m on.
static __device__ __noinline__ Pair pair_key(float l, float b, float m, Pair z, bool sigmoid) {
  // exp(l - m); exp(-l), or exp(l)
  const Pair e = pair_exp(!sigmoid ? pair_sum(l, -m) : Pair{-fabsf(l), 0.0f});
  const Pair one = {1.0f, 0.0f};
  Pair above = e, below = z;
  if (sigmoid) {
    below = one + e;
    if (l > 0.0f) above = one;
  }
  return over(above, below) + Pair{b, 0.0f};
}

__device__ __forceinline__ Pair pair_lane(Pair r, uint32_t mask, int lane) {
  return {__shfl_sync(mask, r.hi, lane), __shfl_sync(mask, r.lo, lane)};
}

// The sum of a row's exponentials from the largest logit on, by the row's lanes.
template <int TYPE, int LANES>
__device__ __noinline__ Pair route_pair_z(const RouteParams& p, int64_t row, int first, int count, float m,
                                          uint32_t mask) {
  Pair z = {0.0f, 0.0f};
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    const float l = route_load<TYPE>(p.logits, row * p.ld + first + j);
    z = z + pair_exp(pair_sum(l, -m));
  }
  for (int o = LANES / 2; o > 0; o >>= 1) z = z + pair_lane(z, mask, static_cast<int>(lane_id()) ^ o);
  return z;
}

// Whether a differs from b by more than the Pairs' errors (2^-40 of the keys' size, where
// that is not so small that Pairs lose bits).
__device__ __forceinline__ bool pairs_apart(Pair a, Pair b, float b_most) {
  const float size = fmaxf(fabsf(a.hi), fabsf(b.hi)) + b_most;
  return size > 0x1p-70f && fabsf((a.hi - b.hi) + (a.lo - b.lo)) > 0x1p-40f * size;
}

// Which of two groups has the larger sum of its two best scores, by their logits a1 >= a2
// and b1 >= b2 (-infinity: none): 1 the first, -1 the second, 0 neither. Scores f rise with
// their logits, so that only a1 > b1 >= b2 > a2 (or the reverse) is a question: whether
// f(a1) - f(b1) > f(b2) - f(a2). Both differences are products of positive factors,
//
//   softmax:  f(x) - f(y) = exp(x) (1 - exp(y - x))             (the row's sum left out)
//   sigmoid:  f(x) - f(y) = f(x) f(-y) (1 - exp(y - x)),   f(x) = exp(min(x, 0)) / (1 + exp(-|x|))
//
// and the logarithm of their quotient, the powers of e put together, is compared with 0: no
// score is too small for it, and none too near 1. In 32 bits if it is far enough from 0, else in
// 64. (32 bits: 22 roundings of 2^-24 in the quotient, and in the powers and the logarithm,
// which cancel, five of their size.)
template <typename F>
__device__ __forceinline__ F sums_quotient(F a1, F a2, F b1, F b2, bool sigmoid, F& size) {
  const F zero = 0, one = 1;
  F power = a1 - b2, quotient = expm1(b1 - a1) / expm1(a2 - b2);
  size = power;
  if (sigmoid) {
    const F up = fmin(a1, zero) - fmin(b2, zero), down = fmax(b1, zero) - fmax(a2, zero);  // (both >= 0)
    power = up - down;
    size = up + down;
    quotient *= ((one + exp(-fabs(b2))) * (one + exp(-fabs(a2)))) / ((one + exp(-fabs(a1))) * (one + exp(-fabs(b1))));
  }
  return power + log(quotient);
}
static __device__ __noinline__ int compare_sums(float a1, float a2, float b1, float b2, bool sigmoid) {
  if (a1 == b1) return (a2 > b2) - (a2 < b2);
  int sign = 1;
  if (a1 < b1) {
    const float t1 = a1, t2 = a2;
    a1 = b1;
    a2 = b2;
    b1 = t1;
    b2 = t2;
    sign = -1;
  }
  if (a2 >= b2) return sign;
  float size;
  const float near = sums_quotient<float>(a1, a2, b1, b2, sigmoid, size);
  if (fabsf(near) > 0x1p-18f + 0x1p-20f * size && fabsf(near) < INFINITY) return near > 0.0f ? sign : -sign;
  double size64;
  const double exact = sums_quotient<double>(a1, a2, b1, b2, sigmoid, size64);
  return exact > 0.0 ? sign : exact < 0.0 ? -sign : 0;
}

// The choice of one row in doubt without a bias, by the row's lanes: this lane's pick (lane i has
// the i-th), or -1. It reads its logits anew, as route_careful does.
template <int TYPE, int LANES, int PER>
__device__ __noinline__ int route_by_logits(const RouteParams& p, int64_t row, int first, int count, uint32_t mask) {
  const int sub = static_cast<int>(lane_id()) & (LANES - 1), g = sub >> p.lanes_log2;
  float l[PER], l1 = -INFINITY, l2 = -INFINITY;  // the group's two best
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    l[j] = j < count && !(p.bias && p.bias[first + j] == -INFINITY)
               ? route_load<TYPE>(p.logits, row * p.ld + first + j) : -INFINITY;
    l2 = fmaxf(l2, fminf(l1, l[j]));
    l1 = fmaxf(l1, l[j]);
  }
  bool kept = true;
  if (p.groups > 1) {
    for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
      const float a1 = __shfl_xor_sync(mask, l1, o), a2 = __shfl_xor_sync(mask, l2, o);
      l2 = fmaxf(fminf(l1, a1), fmaxf(l2, a2));
      l1 = fmaxf(l1, a1);
    }
    if (p.group_best == 1) l2 = -INFINITY;
    // most sums lie far enough apart for 32 bits: a softmax's scores from the row's best on
    const float m = from_order_bits(route_max<LANES>(order_bits(l1 + 0.0f), mask));
    const auto score = [&](float v) { return p.sigmoid ? logistic(v) : v > -INFINITY ? expf(v - m) : 0.0f; };
    const float sum = score(l1) + score(l2);
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < p.groups; ++o) {
      const float o1 = __shfl_sync(mask, l1, o << p.lanes_log2, LANES);
      const float o2 = __shfl_sync(mask, l2, o << p.lanes_log2, LANES);
      const float other = __shfl_sync(mask, sum, o << p.lanes_log2, LANES), most = fmaxf(sum, other);
      int sign = other > sum ? 1 : -1;
      if (!(most > 0x1p-100f && fabsf(other - sum) > 0x1p-16f * most))
        sign = compare_sums(o1, o2, l1, l2, p.sigmoid);
      rank += sign > 0 || (sign == 0 && o < g);
    }
    kept = rank < p.top_groups;
  }
  int mine = -1;
  uint32_t taken = 0, taken2 = 0;  // the lane's experts that were picked
#pragma unroll 1
  for (int i = 0; i < p.top; ++i) {
    float best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const bool free = kept && !(((j < 32 ? taken : taken2) >> (j & 31)) & 1u);
      if (free && l[j] > best) {
        best = l[j];
        at = j;
      }
    }
    // (of equal ones the first lane's, whose experts come first)
    const uint32_t key = at >= 0 ? order_bits(best + 0.0f) : 0u;
    const uint32_t most = route_max<LANES>(key, mask);
    if (most == 0) break;
    const uint32_t having = __ballot_sync(mask, key == most);
    const int from = __ffs(having) - 1;
    const int expert = __shfl_sync(mask, first + at, from);
    if (sub == i) mine = expert;
    if (static_cast<int>(lane_id()) == from) {
      if (at < 32)
        taken |= 1u << at;
      else
        taken2 |= 1u << (at & 31);
    }
  }
  return mine;
}

// The choice of one row in 64 bits, by the row's lanes: this lane's pick (lane i
// has the i-th), or -1. For the rows with a bias that even Pairs do not settle (and that have
// more than 16 experts a lane). It reads its inputs anew and holds nothing in the fast
// path's registers.
template <int TYPE, int LANES, int PER>
__device__ __noinline__ int route_careful(const RouteParams& p, int64_t row, int first, int count,
                                          uint32_t mask) {
  const int sub = static_cast<int>(lane_id()) & (LANES - 1);
  const int g = sub >> p.lanes_log2;
  double key[PER];
  double m = -INFINITY;
#pragma unroll 1
  for (int j = 0; j < PER; ++j) {
    key[j] = j < count ? route_load<TYPE>(p.logits, row * p.ld + first + j) : -INFINITY;
    m = fmax(m, key[j]);
  }
  for (int o = LANES / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(mask, m, o));
  double z = 1.0;
  if (!p.sigmoid) {
    z = 0.0;
#pragma unroll 1
    for (int j = 0; j < PER; ++j)
      if (key[j] > -INFINITY) z += exp(key[j] - m);
    for (int o = LANES / 2; o > 0; o >>= 1) z += __shfl_xor_sync(mask, z, o);
  }
  double t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll 1
  for (int j = 0; j < PER; ++j) {
    if (!(key[j] > -INFINITY)) continue;
    const float b = p.bias[first + j];
    if (b == -INFINITY) {
      key[j] = -INFINITY;
      continue;
    }
    const double k = (p.sigmoid ? 1.0 / (1.0 + exp(-key[j])) : exp(key[j] - m) / z) + static_cast<double>(b);
    key[j] = k;
    t2 = fmax(t2, fmin(t1, k));
    t1 = fmax(t1, k);
  }
  if (p.groups > 1) {
    for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
      const double a1 = __shfl_xor_sync(mask, t1, o), a2 = __shfl_xor_sync(mask, t2, o);
      t2 = fmax(fmin(t1, a1), fmax(t2, a2));
      t1 = fmax(t1, a1);
    }
    const double sum = p.group_best == 2 && t2 > -INFINITY ? t1 + t2 : t1;
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const double other = __shfl_sync(mask, sum, o << p.lanes_log2, LANES);
      rank += other > sum || (other == sum && o < g);
    }
    if (rank >= p.top_groups)
      for (int j = 0; j < PER; ++j) key[j] = -INFINITY;
  }
  int mine = -1;
  for (int i = 0; i < p.top; ++i) {
    double best = -INFINITY;
    int at = INT32_MAX;
#pragma unroll 1
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
    if (at >= first && at < first + PER) key[at - first] = -INFINITY;
  }
  return mine;
}

// (Seven blocks an SM: 32768 rows of 256 experts, 8 groups 36.3 us, of 64 experts 8.8 us; six 38.0
// and 9.0 us, eight 36.3 and 9.2 us.)
template <int TYPE, int LANES, int PER>
__global__ void __launch_bounds__(32 * ROUTE_WARPS, PER == 8 ? 7 : 1)
    route_experts_kernel(const __grid_constant__ RouteParams p) {
  constexpr int N = TYPE == ROUTE_F32 ? 4 : 8;  // logits in 16 bytes
  constexpr uint32_t PLACE = PER - 1;           // a key's lowest bits: PER - 1 - place in the lane
  constexpr int AT_ONCE = 32 / LANES;           // rows of a turn
  constexpr bool SORTED = PER <= 16;            // (more keys: the largest is looked for each time)
  constexpr uint32_t ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31, sub = lane & (LANES - 1);
  const uint32_t mask = LANES == 32 ? ALL : ((1u << (LANES & 31)) - 1u) << (lane - sub);
  const int64_t row0 =
      (static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS + (threadIdx.x >> 5)) * AT_ONCE * p.turns;
  if (row0 >= p.rows) return;
  const int g = sub >> p.lanes_log2, q = sub & ((1 << p.lanes_log2) - 1);
  const int first = g * p.size + q * p.chunk;
  const int count = g < p.groups ? max(0, min(p.chunk, p.size - q * p.chunk)) : 0;
  grid_dependency_wait();

  // The bias: the same for all rows.
  float b[PER];
  float b_most = 0.0f;  // the largest by magnitude, of experts that can be chosen
  bool b_nan = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) b[j] = 0.0f;
  if (p.bias != nullptr) {
    if (p.wide_bias) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i)
        if (4 * i < count) {
          const float4 v = *reinterpret_cast<const float4*>(p.bias + first + 4 * i);
          b[4 * i] = v.x;
          b[4 * i + 1] = v.y;
          b[4 * i + 2] = v.z;
          b[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j < count) b[j] = p.bias[first + j];
    }
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (b[j] != -INFINITY) most = max(most, __float_as_uint(b[j]) & 0x7fffffffu);
    b_most = __uint_as_float(__reduce_max_sync(ALL, most));
    b_nan = b_most != b_most;
  }
  // Whether logits stand for the keys: exactly, if they have 16 bits.
  const bool biased = b_most != 0.0f;
  const bool direct = !biased && (p.groups == 1 || p.group_best == 1);
  const bool exact = direct && TYPE != ROUTE_F32;

  // One place of a row's picks, by lane: the expert (-1: none, -2: the
  // row's weights are NaN), whether the row is in doubt, and for a softmax the largest
  // logit and the reciprocal of the sum.
  int pick = -1;
  bool doubt = false;
  float my_m = 0.0f, my_rz = 1.0f;
  const int slots = 1 << p.slots_log2;
  const int my_row = lane >> p.slots_log2, my_slot = lane & (slots - 1);

  for (int turn = 0; turn < p.turns; ++turn) {
    const int64_t at = row0 + turn * AT_ONCE + lane / LANES;
    if (row0 + turn * AT_ONCE >= p.rows) break;
    const int64_t row = min(at, p.rows - 1);  // (lanes past the end repeat the last row)
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
    float m = max_nan(l[0], l[1], l[2]);
#pragma unroll
    for (int j = 3; j + 1 < PER; j += 2) m = max_nan(m, l[j], l[j + 1]);
    m = max_nan(m, m, l[PER - 1]);
    bool bad = b_nan || m != m || (!p.sigmoid && m == INFINITY);
    bad = (__ballot_sync(ALL, bad) & mask) != 0;
    uint32_t k[PER];
    float rz = 1.0f;
    if (p.sigmoid) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float key = l[j] + 0.0f;
        if (!direct) key = logistic_key(l[j]) + b[j];
        k[j] = order_bits(key);
      }
    } else {
      m = from_order_bits(route_max<LANES>(order_bits(m + 0.0f)));
      float e[PER];
      if (!p.renorm || !direct) {
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          e[j] = l[j] > -INFINITY ? expf(l[j] - m) : 0.0f;
          z += e[j];
        }
        rz = 1.0f / route_sum<LANES>(z);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) k[j] = order_bits(direct ? l[j] + 0.0f : e[j] * rz + b[j]);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      k[j] = l[j] > -INFINITY && b[j] != -INFINITY ? (k[j] & ~PLACE) | (PLACE - j) : 0u;
    if constexpr (SORTED) sort_down<0, PER>(k);
    bool unsettled = false;
    // what scores are divided by, as a Pair: a softmax's sum beside a bias, once it has been needed
    Pair z2 = {1.0f, 0.0f};
    bool summed = p.sigmoid;
    if (p.groups > 1) {
      uint32_t t1 = 0, t2 = 0;
      if constexpr (SORTED) {
        t1 = k[0];
        t2 = k[1];
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          t2 = max(t2, min(t1, k[j]));
          t1 = max(t1, k[j]);
        }
      }
      for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
        const uint32_t a1 = __shfl_xor_sync(ALL, t1, o), a2 = __shfl_xor_sync(ALL, t2, o);
        t2 = max(min(t1, a1), max(t2, a2));
        t1 = max(t1, a1);
      }
      uint32_t score = t1 & ~PLACE;
      if (p.group_best == 2 && t2 != 0)
        score = order_bits(from_order_bits(t1 & ~PLACE) + from_order_bits(t2 & ~PLACE) + 0.0f);
      // (groups after the last have lanes of count 0: score 0, behind all others)
      int rank = 0;
      for (int o0 = 0; o0 < p.groups; o0 += 1 << p.lanes_log2) {  // (each lane of a group looks at others)
        const int o = o0 + q;
        const uint32_t other = __shfl_sync(ALL, score, o << p.lanes_log2, LANES);
        rank += o < p.groups && (other > score || (other == score && o < g));
      }
      for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) rank += __shfl_xor_sync(ALL, rank, o);
      bool kept = rank < p.top_groups;
      if (!exact) {
        const float w = from_order_bits(~route_max<LANES>(kept ? ~score : 0u));
        const uint32_t next = route_max<LANES>(kept ? 0u : score);
        const bool near = next != 0 && !(w - from_order_bits(next) >
                                         2.0f * route_apart<PER>(w, 4.0f * b_most, p.sigmoid));
        if (near && (!biased || !SORTED)) {
          unsettled = true;
        } else if (near) {
          if constexpr (SORTED) {
            // the groups' sums anew, from each lane's two best keys
            if (!summed) z2 = route_pair_z<TYPE, LANES>(p, row, first, count, m, mask);
            summed = true;
            Pair d[2];
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const uint32_t c = i ? k[1] : k[0];
              const int e = first + static_cast<int>(PLACE - (c & PLACE));
              const float el = c ? route_load<TYPE>(p.logits, row * p.ld + e) : 0.0f;
              const float eb = c && p.bias ? p.bias[e] : 0.0f;
              const Pair v = pair_key(el, eb, m, z2, p.sigmoid);
              (i ? d[1] : d[0]) = c ? v : Pair{-INFINITY, 0.0f};
            }
            // A lane's third key near its second might be its second, unless it is a tie with it.
            const float second = from_order_bits(k[1] & ~PLACE);
            const float apart = route_apart<PER>(second, b_most, p.sigmoid);
            const int e1 = first + static_cast<int>(PLACE - (k[1] & PLACE));
#pragma unroll
            for (int j = 2; j < PER; ++j)
              if (k[j] != 0 && !(second - from_order_bits(k[j] & ~PLACE) > apart)) {
                const int e = first + static_cast<int>(PLACE - (k[j] & PLACE));
                if (route_load<TYPE>(p.logits, row * p.ld + e) != route_load<TYPE>(p.logits, row * p.ld + e1) ||
                    (p.bias && p.bias[e] != p.bias[e1]))
                  unsettled = true;
              }
            if (d[1] > d[0]) {
              const Pair v = d[0];
              d[0] = d[1];
              d[1] = v;
            }
            for (int o = 1; o < (1 << p.lanes_log2); o <<= 1) {
              const Pair a1 = pair_lane(d[0], mask, lane ^ o), a2 = pair_lane(d[1], mask, lane ^ o);
              const Pair low = a1 > d[0] ? d[0] : a1, high = a2 > d[1] ? a2 : d[1];
              d[1] = low > high ? low : high;
              d[0] = a1 > d[0] ? a1 : d[0];
            }
            const Pair sum = p.group_best == 2 && d[1].hi > -INFINITY ? d[0] + d[1] : d[0];
            rank = 0;
#pragma unroll 1
            for (int o = 0; o < p.groups; ++o) {
              const int at = (lane - sub) + (o << p.lanes_log2);
              const Pair other = pair_lane(sum, mask, at);
              rank += other > sum || (other == sum && o < g);
              // (of the same two keys: a tie, as between groups of a row of zeros)
              const Pair other1 = pair_lane(d[0], mask, at), other2 = pair_lane(d[1], mask, at);
              const bool tie = other1 == d[0] && other2 == d[1];
              // (a sum past the largest float is infinite or NaN, and settles nothing)
              if (o != g && g < p.groups && sum.hi != -INFINITY && other.hi != -INFINITY && !tie &&
                  !pairs_apart(sum, other, 4.0f * b_most))
                unsettled = true;
            }
            kept = rank < p.top_groups;
          }
        }
      }
      if (!kept) {
#pragma unroll
        for (int j = 0; j < PER; ++j) k[j] = 0;
      }
    }
    // The picks: lane i keeps the i-th key and the lane that it came from.
    uint32_t best = k[0], key = 0, own_key = 0;
    if constexpr (!SORTED) {
#pragma unroll
      for (int j = 1; j < PER; ++j) best = max(best, k[j]);
    }
    int own_from = 0, from = 0;
    for (int i = 0; i < p.top; ++i) {
      const uint32_t most = route_max<LANES>(best & ~PLACE);
      from = __ffs(__ballot_sync(ALL, (best & ~PLACE) == most) & mask) - 1;  // (the lowest of a tie)
      key = __shfl_sync(ALL, best, from);
      if (sub == i) {
        own_key = key;
        own_from = from;
      }
      if constexpr (SORTED) {
        if (lane == from) {
#pragma unroll
          for (int j = 1; j < PER; ++j) k[j - 1] = k[j];
          k[PER - 1] = 0;
        }
        best = k[0];
      } else if (lane == from) {
        best = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          k[j] = k[j] == key ? 0u : k[j];
          best = max(best, k[j]);
        }
      }
    }
    const auto expert_of = [&](uint32_t key, int from) {
      const int s = from & (LANES - 1);
      return (s >> p.lanes_log2) * p.size + (s & ((1 << p.lanes_log2) - 1)) * p.chunk +
             static_cast<int>(PLACE - (key & PLACE));
    };
    int own = own_key != 0 ? expert_of(own_key, own_from) : -1;
    if (!exact) {
      // A pick near the next one, or an expert that was not picked near the last pick.
      const uint32_t next_key = __shfl_down_sync(ALL, own_key, 1, LANES);
      const float own_f = from_order_bits(own_key & ~PLACE), last_f = from_order_bits(key & ~PLACE);
      const float last_apart = direct ? 0.0f : route_apart<PER>(last_f, b_most, p.sigmoid);
      const auto near_last = [&](uint32_t k) {
        return k != 0 && key != 0 && !(last_f - from_order_bits(k & ~PLACE) > last_apart);
      };
      bool near = sub + 1 < p.top && next_key != 0 &&
                  !(own_f - from_order_bits(next_key & ~PLACE) >
                    (direct ? 0.0f : route_apart<PER>(own_f, b_most, p.sigmoid)));
      const bool extra = near_last(best);
      if ((__ballot_sync(ALL, near || extra) & mask) != 0 && !bad) {
        // Not if it is a tie with the same logit and bias.
        const int base = lane - sub;
        const int mine_e = extra ? first + static_cast<int>(PLACE - (best & PLACE)) : -1;
        const float ol = own >= 0 ? route_load<TYPE>(p.logits, row * p.ld + own) : 0.0f;
        const float ob = own >= 0 && p.bias ? p.bias[own] : 0.0f;
        const float el = extra ? route_load<TYPE>(p.logits, row * p.ld + mine_e) : 0.0f;
        const float eb = extra && p.bias ? p.bias[mine_e] : 0.0f;
        const float nl = __shfl_down_sync(mask, ol, 1, LANES), nb = __shfl_down_sync(mask, ob, 1, LANES);
        const float ll = __shfl_sync(mask, ol, base + p.top - 1), lb = __shfl_sync(mask, ob, base + p.top - 1);
        if (near && ol == nl && ob == nb) near = false;
        // (and all others of the lane that lie as near)
        bool differs = extra && (el != ll || eb != lb), others = false, others_differ = false;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (k[j] != best && near_last(k[j])) {
            const int e = first + static_cast<int>(PLACE - (k[j] & PLACE));
            others = true;
            others_differ = others_differ || route_load<TYPE>(p.logits, row * p.ld + e) != ll ||
                            (p.bias && p.bias[e] != lb);
          }
        const bool rank = __ballot_sync(mask, near || differs || others_differ) != 0;
        // (ranked is one expert a lane beside the picks, and none of unsorted keys)
        unsettled = unsettled || (rank && (others || !SORTED || !biased));
        if (SORTED && rank && biased) {
          // The picks and the extra ones, ranked by Pairs.
          if (!summed) z2 = route_pair_z<TYPE, LANES>(p, row, first, count, m, mask);
          const Pair none = {-INFINITY, 0.0f};
          Pair a = pair_key(ol, ob, m, z2, p.sigmoid), c = none;
          if (own < 0) a = none;
          const uint32_t extras = __ballot_sync(mask, extra);
          if (extras != 0) c = pair_key(el, eb, m, z2, p.sigmoid);
          if (!extra) c = none;
          int rank_a = 0, rank_c = 0;
          const auto against = [&](Pair v, int e, float vl, float vb) {
            if (e < 0) return;
            rank_a += v > a || (v == a && e < own);
            rank_c += v > c || (v == c && e < mine_e);
            if (own >= 0 && e != own && !pairs_apart(v, a, b_most) && (vl != ol || vb != ob))
              unsettled = true;
            if (extra && e != mine_e && !pairs_apart(v, c, b_most) && (vl != el || vb != eb))
              unsettled = true;
          };
#pragma unroll 1
          for (int i = 0; i < p.top; ++i)
            against(pair_lane(a, mask, base + i), __shfl_sync(mask, own, base + i), __shfl_sync(mask, ol, base + i),
                    __shfl_sync(mask, ob, base + i));
#pragma unroll 1
          for (uint32_t left = extras; left != 0; left &= left - 1) {
            const int from_e = __ffs(left) - 1;
            against(pair_lane(c, mask, from_e), __shfl_sync(mask, mine_e, from_e), __shfl_sync(mask, el, from_e),
                    __shfl_sync(mask, eb, from_e));
          }
          int ranked = -1;
#pragma unroll 1
          for (int i = 0; i < p.top; ++i) {
            const int e = __shfl_sync(mask, own, base + i), r = __shfl_sync(mask, rank_a, base + i);
            if (e >= 0 && r == sub) ranked = e;
          }
#pragma unroll 1
          for (uint32_t left = extras; left != 0; left &= left - 1) {
            const int e = __shfl_sync(mask, mine_e, __ffs(left) - 1), r = __shfl_sync(mask, rank_c, __ffs(left) - 1);
            if (r == sub) ranked = e;
          }
          own = sub < p.top ? ranked : -1;
        }
      }
    }
    unsettled = (__ballot_sync(ALL, unsettled) & mask) != 0 && !bad;
    // to the lanes of the row's places
    if (bad) own = -2;
    own = (own + 2) | (unsettled ? 1 << 16 : 0);
    const int source = (my_row & (AT_ONCE - 1)) * LANES + my_slot;
    const int got = __shfl_sync(ALL, own, source);
    float got_m = 0.0f, got_rz = 1.0f;
    if (!p.renorm) {
      got_m = __shfl_sync(ALL, m, source);
      got_rz = __shfl_sync(ALL, rz, source);
    }
    if (my_row / AT_ONCE == turn) {
      pick = my_slot < p.top ? (got & 0xffff) - 2 : -1;
      doubt = (got >> 16) != 0;
      my_m = got_m;
      my_rz = got_rz;
    }
  }

  const bool live = my_slot < p.top && my_row < AT_ONCE * p.turns && row0 + my_row < p.rows;
  const int64_t row = min(row0 + my_row, p.rows - 1);
  float my_l = pick >= 0 ? route_load<TYPE>(p.logits, row * p.ld + pick) : -INFINITY;
  if (!exact) {
    const uint32_t doubts = __ballot_sync(ALL, doubt && live);
    for (int r = 0; doubts != 0 && r < 32 >> p.slots_log2; ++r) {
      if (((doubts >> (r << p.slots_log2)) & ((1u << slots) - 1u)) == 0) continue;
      // (with fewer lanes a row than a warp has, all of the warp's parts do the same)
      const int careful = biased ? route_careful<TYPE, LANES, PER>(p, row0 + r, first, count, mask)
                                 : route_by_logits<TYPE, LANES, PER>(p, row0 + r, first, count, mask);
      const int found = __shfl_sync(ALL, careful, my_slot);
      if (my_row == r) {
        pick = my_slot < p.top ? found : -1;
        my_l = pick >= 0 ? route_load<TYPE>(p.logits, row * p.ld + pick) : -INFINITY;
      }
    }
  }
  // The weights. Renormalised ones relative to the largest chosen score, so that
  // scores that all lie near zero keep their ratios.
  float w;
  if (p.renorm) {
    uint32_t most = pick >= 0 ? order_bits(my_l + 0.0f) : 0u;
    for (int o = slots / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(ALL, most, o));
    const float ref = from_order_bits(most);
    float d = my_l - ref;
    if (p.sigmoid)
      d = (fminf(my_l, 0.0f) - fminf(ref, 0.0f)) - (log1pf(expf(-fabsf(my_l))) - log1pf(expf(-fabsf(ref))));
    w = pick >= 0 ? expf(d) : 0.0f;
    float total = w;
    for (int o = slots / 2; o > 0; o >>= 1) total += __shfl_xor_sync(ALL, total, o);
    w = pick >= 0 ? w / total : 0.0f;
  } else {
    w = pick < 0 ? 0.0f : p.sigmoid ? logistic(my_l) : expf(my_l - my_m) * my_rz;
  }
  w *= p.scale;
  if (pick == -2) {
    pick = my_slot;
    w = NAN;
  }
  if (live) {
    p.weights[row * p.top + my_slot] = w;
    p.experts[row * p.top + my_slot] = pick;
  }
  grid_launch_dependents();
}

// Gradient of the logits, SLOTS lanes (8 or 16, one a pick) to a row. With c the chosen experts, g the
// weights' gradient times scale:
//
//   sigmoid               d_c = g_c s_c (1 - s_c)
//   sigmoid, renormalised d_c = (g_c - sum g u) u_c (1 - s_c)      u: renormalised scores
//   softmax, renormalised d_c = (g_c - sum g u) u_c
//   softmax               d_e = s_e ([e chosen] g_e - sum g s)      for every expert
//
// Only the last reads all logits. The row is written first (zeros, or -s sum g s),
// then the chosen experts' values over it.
template <int TYPE, int SLOTS>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
    route_experts_dlogits_kernel(const __grid_constant__ RouteGradParams p) {
  constexpr int N = TYPE == ROUTE_F32 ? 4 : 8;
  constexpr int OUT = TYPE == ROUTE_F32 ? OUT_F32 : TYPE == ROUTE_BF16 ? OUT_BF16 : OUT_F16;
  const int lane = threadIdx.x & (SLOTS - 1);
  constexpr uint32_t ALL = 0xffffffffu;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * ROUTE_WARPS * 32 + threadIdx.x) / SLOTS;
  const int64_t row = min(at, p.rows - 1);  // (lanes past the end repeat the last row and store nothing)
  grid_dependency_wait();
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
      for (int i = lane; i < p.E / N; i += SLOTS) {
        float v[N];
        route_unpack<TYPE>(reinterpret_cast<const uint4*>(src)[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
      }
    } else {
      for (int i = lane; i < p.E; i += SLOTS) m = fmaxf(m, route_load<TYPE>(src, i));
    }
#pragma unroll
    for (int o = SLOTS / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(ALL, m, o));
    if (p.wide) {
      for (int i = lane; i < p.E / N; i += SLOTS) {
        float v[N];
        route_unpack<TYPE>(reinterpret_cast<const uint4*>(src)[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) z += v[j] == -INFINITY ? 0.0f : expf(v[j] - m);
      }
    } else {
      for (int i = lane; i < p.E; i += SLOTS) {
        const float v = route_load<TYPE>(src, i);
        z += v == -INFINITY ? 0.0f : expf(v - m);
      }
    }
    rz = 1.0f / route_sum<SLOTS>(z);
  }
  // scores of the chosen (u: those that the weights are) and the sum of g u
  float s = 0.0f, u;
  if (p.renorm) {
    const float ref = from_order_bits(route_max<SLOTS>(e >= 0 ? order_bits(l + 0.0f) : 0u));
    float x = l - ref;
    if (p.sigmoid) {
      s = logistic(l);
      x = (fminf(l, 0.0f) - fminf(ref, 0.0f)) - (log1pf(expf(-fabsf(l))) - log1pf(expf(-fabsf(ref))));
    }
    u = e >= 0 ? expf(x) : 0.0f;
    const float total = route_sum<SLOTS>(u);
    u = e >= 0 ? u / total : 0.0f;
  } else {
    u = e < 0 ? 0.0f : p.sigmoid ? logistic(l) : l == -INFINITY ? 0.0f : expf(l - m) * rz;
    s = u;
  }
  const float dot = p.sigmoid && !p.renorm ? 0.0f : route_sum<SLOTS>(g * u);
  // an expert named twice gets both gradients (its score stands twice in the sums)
  float own = 0.0f;
  for (int i = 0; i < p.top; ++i) {
    const int oe = __shfl_sync(ALL, e, i, SLOTS);
    const float og = __shfl_sync(ALL, g, i, SLOTS);
    if (oe == e) own += p.renorm ? og - dot : og;
  }
  float d = own * u;
  if (full) d = u * (own - dot);
  // 1 - s, without cancellation
  if (p.sigmoid) d *= logistic(-l);
  const float back = full ? -dot : 0.0f;
  if (at < p.rows && p.wide) {
    for (int i = lane; i < p.E / N; i += SLOTS) {
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
  } else if (at < p.rows) {
    for (int i = lane; i < p.E; i += SLOTS) {
      float v = 0.0f;
      if (full) {
        v = route_load<TYPE>(src, i);
        v = v == -INFINITY ? 0.0f : expf(v - m) * rz * back;
      }
      store_out<OUT>(dst, i, v);
    }
  }
  __syncwarp();  // (orders the row's stores before those of the chosen)
  if (e >= 0 && at < p.rows) store_out<OUT>(dst, e, d);
  grid_launch_dependents();
}

}  // namespace sptg
