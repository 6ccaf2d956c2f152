// add_rms_norm.cuh -- residual addition and root-mean-square norm of each row,
// with an 8-bit output and a scale for each row (or a 16-bit output).
//
//   h = x + r                              (32 bits; rounded once to the 16-bit residual out)
//   y = h * w / sqrt(mean(h^2) + eps)
//   s = max|y| / QMAX,  q = round(y / s)   (QMAX = 127 for int8, 448 for e4m3)
//
// The reciprocal root is the same for a whole row, so max|y| = rstd * max|h w|
// and y / s = h w * (QMAX / max|h w|): the sum of squares and the maximum come
// out of one pass over the row and one exchange between its threads, and the
// quantised values never depend on the reciprocal root.
//
// A row with an infinite or NaN h (or w) gets q = 0 and s = NaN, so that every
// value it stands for is NaN; one whose max|h w| is zero, or so small that
// QMAX / max|h w| overflows, or whose finite h are so large that their squares
// overflow (y is 0 by the formula), gets q = 0 and s = 0. The maximum of |h| is
// kept beside that of |h w| to tell an overflow from an infinity.
//
// Memory-bound: 7 bytes an element (x, r in; h, q out) and some ten flops. The
// row stays in registers between the reduction and the outputs (32 elements a
// thread), so x and r are read once.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sptg {

// Output kinds: 8-bit with row scales, or the input's own 16-bit type.
enum NormOut : int { NORM_S8 = 0, NORM_E4M3 = 1, NORM_16 = 2 };

struct NormParams {
  const void* x;
  const void* r;
  const void* w;
  void* h;
  void* q;
  float* scales;
  int64_t ldx, ldr, ldh, ldq;  // elements between rows
  int64_t rows;
  int cols;
  float eps;
};

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

template <bool BF16>
__device__ __forceinline__ float load16(const void* p, int64_t i) {
  if constexpr (BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else
    return __half2float(static_cast<const __half*>(p)[i]);
}

// Two values to the 8-bit type, in the low 16 bits (lo at the lower address).
template <int OUTK>
__device__ __forceinline__ uint32_t quant2(float lo, float hi) {
  if constexpr (OUTK == NORM_S8) {
    // round to nearest even, then clamp (the scaled value passes 127 by
    // rounding errors at most)
    const int a = max(-127, min(127, __float2int_rn(lo)));
    const int b = max(-127, min(127, __float2int_rn(hi)));
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
  } else {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  }
}

// What a row's statistics leave for its elements: q = h w * qmul (0 when
// `zero`), y = h * rstd * w.
struct RowScale {
  float rstd, qmul, scale;
  bool zero;
};

// Maxima are held as the bits of non-negative floats and compared as unsigned
// integers, so that NaN (above every number) is kept. mx: .x max|h w|, .y max|h|.
template <int OUTK>
__device__ __forceinline__ RowScale row_scale(float sumsq, uint2 mx, int cols, float eps) {
  RowScale s;
  s.rstd = 1.0f / sqrtf(sumsq / static_cast<float>(cols) + eps);
  constexpr float QMAX = OUTK == NORM_S8 ? 127.0f : 448.0f;
  const float m = __uint_as_float(mx.x);
  s.qmul = QMAX / m;
  const bool overflow = !(s.rstd > 0.0f) && __uint_as_float(mx.y) < INFINITY;
  const bool bad = !(m < INFINITY) && !overflow;
  s.zero = bad || overflow || !(s.qmul < INFINITY);
  s.scale = bad ? NAN : s.zero ? 0.0f : s.rstd * m / QMAX;
  return s;
}

// Sum and maxima over the `TPR` threads of a row, the same for each of them.
// The order of the sum is fixed: lanes by halves, then warps in turn.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, uint2& mx, float* s_sum, uint2* s_max,
                                           int row_slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  mx.x = __reduce_max_sync(0xffffffffu, mx.x);
  mx.y = __reduce_max_sync(0xffffffffu, mx.y);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
      s_sum[warp] = sum;
      s_max[warp] = mx;
    }
    __syncthreads();
    sum = 0.0f;
    mx = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sum += s_sum[row_slot * W + i];
      mx.x = max(mx.x, s_max[row_slot * W + i].x);
      mx.y = max(mx.y, s_max[row_slot * W + i].y);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Rows of up to TPR * PER * 8 elements held in registers; THREADS / TPR rows
// to a block. Needs 16-byte aligned rows and cols a multiple of 8.
template <bool BF16, int OUTK, int TPR, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) add_rms_norm_kernel(const NormParams p) {
  __shared__ float s_sum[THREADS / 32];
  __shared__ uint2 s_max[THREADS / 32];
  const int slot = threadIdx.x / TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / TPR) + slot;
  const bool live = row < p.rows;
  const int groups = p.cols >> 3;  // groups of 8 elements
  // a block of 1024 threads has 64 registers for each: it reads w a second
  // time (from L1) instead of keeping it
  constexpr bool KEEP_W = THREADS < 1024;
  grid_dependency_wait();
  uint4 xv[PER], rv[PER], wv[PER];
  const uint4* px = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.ldx);
  const uint4* pr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.r) + row * p.ldr);
  const uint4* pw = static_cast<const uint4*>(p.w);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = lane + i * TPR;
    const bool in = live && g < groups;
    xv[i] = in ? __ldcs(px + g) : make_uint4(0, 0, 0, 0);  // read once
    rv[i] = in ? __ldcs(pr + g) : make_uint4(0, 0, 0, 0);
    wv[i] = in ? __ldg(pw + g) : make_uint4(0, 0, 0, 0);
  }
  float h[PER][8];
  float sum = 0.0f;
  uint2 mx = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
    const uint32_t rw[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
    const uint32_t ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = unpack2<BF16>(xw[j]), b = unpack2<BF16>(rw[j]), c = unpack2<BF16>(ww[j]);
      const float h0 = a.x + b.x, h1 = a.y + b.y;
      h[i][2 * j] = h0;
      h[i][2 * j + 1] = h1;
      sum += h0 * h0;
      sum += h1 * h1;
      if constexpr (OUTK != NORM_16) {
        mx.x = max(mx.x, max(abs_bits(h0 * c.x), abs_bits(h1 * c.y)));
        mx.y = max(mx.y, max(abs_bits(h0), abs_bits(h1)));
      }
    }
  }
  row_reduce<TPR>(sum, mx, s_sum, s_max, slot);
  grid_launch_dependents();
  if (!live) return;
  const RowScale sc = row_scale<OUTK>(sum, mx, p.cols, p.eps);
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  uint4* ph = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h) + row * p.ldh);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = lane + i * TPR;
    if (g >= groups) continue;
    const float* v = h[i];
    ph[g] = make_uint4(pack2<H_OUT>(v[0], v[1]), pack2<H_OUT>(v[2], v[3]),
                       pack2<H_OUT>(v[4], v[5]), pack2<H_OUT>(v[6], v[7]));
    const uint4 wi = KEEP_W ? wv[i] : __ldg(pw + g);
    const uint32_t ww[4] = {wi.x, wi.y, wi.z, wi.w};
    if constexpr (OUTK == NORM_16) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = unpack2<BF16>(ww[j]);
        o[j] = pack2<H_OUT>(v[2 * j] * sc.rstd * c.x, v[2 * j + 1] * sc.rstd * c.y);
      }
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q) + row * p.ldq)[g] =
          make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = unpack2<BF16>(ww[j]);
        o[j] = sc.zero ? 0u
                       : quant2<OUTK>(v[2 * j] * c.x * sc.qmul, v[2 * j + 1] * c.y * sc.qmul);
      }
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q) + row * p.ldq)[g] =
          make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
  }
  if (OUTK != NORM_16 && lane == 0) p.scales[row] = sc.scale;
}

// Rows of any width, alignment and pitch: one block to a row, element by
// element, x + r formed a second time for the outputs (the second read comes
// from L2). h may be r itself: each element is read by the thread that later
// writes it, in both passes.
template <bool BF16, int OUTK>
__global__ void __launch_bounds__(512) add_rms_norm_any_kernel(const NormParams p) {
  __shared__ float s_sum[16];
  __shared__ uint2 s_max[16];
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx;
  const uint16_t* r = static_cast<const uint16_t*>(p.r) + row * p.ldr;
  float sum = 0.0f;
  uint2 mx = make_uint2(0, 0);
  for (int i = threadIdx.x; i < p.cols; i += 512) {
    const float h = load16<BF16>(x, i) + load16<BF16>(r, i);
    sum += h * h;
    if constexpr (OUTK != NORM_16) {
      mx.x = max(mx.x, abs_bits(h * load16<BF16>(p.w, i)));
      mx.y = max(mx.y, abs_bits(h));
    }
  }
  row_reduce<512>(sum, mx, s_sum, s_max, 0);
  grid_launch_dependents();
  const RowScale sc = row_scale<OUTK>(sum, mx, p.cols, p.eps);
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  for (int i = threadIdx.x; i < p.cols; i += 512) {
    const float h = load16<BF16>(x, i) + load16<BF16>(r, i);
    const float w = load16<BF16>(p.w, i);
    store_out<H_OUT>(p.h, row * p.ldh + i, h);
    if constexpr (OUTK == NORM_16)
      store_out<H_OUT>(p.q, row * p.ldq + i, h * sc.rstd * w);
    else
      static_cast<uint8_t*>(p.q)[row * p.ldq + i] =
          sc.zero ? 0 : static_cast<uint8_t>(quant2<OUTK>(h * w * sc.qmul, 0.0f));
  }
  if (OUTK != NORM_16 && threadIdx.x == 0) p.scales[row] = sc.scale;
}

}  // namespace sptg
