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
// kept beside that of |h w| to tell an overflow from an infinity. Where |h w|
// passes 32 bits although both are finite (bfloat16 only), the row is gone through
// once more with w / 2^64, exact for every product that counts beside one of
// 2^128, and s takes the 2^64 back. (In a loop of its own: scaling the weights
// that the kernels hold costs registers, 16384 rows of 4096 71 -> 80 us.)
//
// Memory-bound: 7 bytes an element (x, r in; h, q out) and some ten flops. The
// row stays in registers (wide rows: in shared memory) between the reduction and
// the outputs, so x and r are read once. 16384 bf16 rows of 8192 to e4m3 155 us,
// 6.1 TB/s, to int8 159 us, to bf16 169 us; of 4096 72 us to e4m3, 76 us to int8;
// 333 rows of 5000: bound by the call from the host.
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
  int stages;  // depth of the ring kernel's ring
  unsigned int* error_word;
  uint64_t timeout_ns;
  int inject_stall;  // test hook of the ring kernel: a block's second row is never copied
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
__device__ __forceinline__ RowScale row_scale(float sumsq, uint2 mx, int cols, float eps,
                                              float unit = 1.0f) {
  RowScale s;
  s.rstd = 1.0f / sqrtf(sumsq / static_cast<float>(cols) + eps);
  constexpr float QMAX = OUTK == NORM_S8 ? 127.0f : 448.0f;
  const float m = __uint_as_float(mx.x);
  s.qmul = QMAX / m;
  const bool overflow = !(s.rstd > 0.0f) && __uint_as_float(mx.y) < INFINITY;
  const bool bad = !(m < INFINITY) && !overflow;
  s.zero = bad || overflow || !(s.qmul < INFINITY);
  s.scale = bad ? NAN : s.zero ? 0.0f : s.rstd * m / QMAX * unit;  // (unit: what h w was divided by)
  return s;
}

// Sum and maxima over a row's threads, the same for each of them: a warp
// (WARP_ROW), or the whole block. The order of the sum is fixed: lanes by
// halves, then warps in turn. s_sum and s_max hold 32 entries.
template <bool WARP_ROW>
__device__ __forceinline__ void row_reduce(float& sum, uint2& mx, float* s_sum, uint2* s_max) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  mx.x = __reduce_max_sync(0xffffffffu, mx.x);
  mx.y = __reduce_max_sync(0xffffffffu, mx.y);
  if constexpr (!WARP_ROW) {
    const int warps = static_cast<int>(blockDim.x) >> 5;
    if ((threadIdx.x & 31) == 0) {
      s_sum[threadIdx.x >> 5] = sum;
      s_max[threadIdx.x >> 5] = mx;
    }
    __syncthreads();
    sum = 0.0f;
    mx = make_uint2(0, 0);
    for (int i = 0; i < warps; ++i) {
      sum += s_sum[i];
      mx.x = max(mx.x, s_max[i].x);
      mx.y = max(mx.y, s_max[i].y);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Whether the products h w of a row of finite h passed 32 bits (or w holds an
// infinity): the same for each of the row's threads.
template <bool BF16, int OUTK>
__device__ __forceinline__ bool products_overflow(uint2 mx) {
  return BF16 && OUTK != NORM_16 && mx.x == 0x7f800000u && mx.y < 0x7f800000u;
}

// What follows a row's statistics, element by element, for any width and
// alignment. x + r is formed once more. h may be x or r itself: each element is
// read by the thread that then writes it. THREADS: of the row, 0 for the block's.
template <bool BF16, int OUTK, int THREADS>
__device__ __forceinline__ void finish_row(const NormParams& p, int64_t row, float sum, uint2 mx,
                                           float* s_sum, uint2* s_max) {
  constexpr bool WARP_ROW = THREADS == 32;
  const int lanes = THREADS ? THREADS : static_cast<int>(blockDim.x);
  const int lane = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx;
  const uint16_t* r = static_cast<const uint16_t*>(p.r) + row * p.ldr;
  float part = 1.0f, unit = 1.0f;  // the weights' part that counts, 1 / part
  if (products_overflow<BF16, OUTK>(mx)) {
    unit = 18446744073709551616.0f;  // 2^64
    part = 1.0f / unit;
    mx.x = 0;
    for (int i = lane; i < p.cols; i += lanes)
      mx.x = max(mx.x, abs_bits((load16<BF16>(x, i) + load16<BF16>(r, i)) * (load16<BF16>(p.w, i) * part)));
    if constexpr (!WARP_ROW) __syncthreads();  // the first sums have been read
    float none = 0.0f;
    row_reduce<WARP_ROW>(none, mx, s_sum, s_max);
  }
  const RowScale sc = row_scale<OUTK>(sum, mx, p.cols, p.eps, unit);
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  for (int i = lane; i < p.cols; i += lanes) {
    const float h = load16<BF16>(x, i) + load16<BF16>(r, i);
    const float w = load16<BF16>(p.w, i);
    store_out<H_OUT>(p.h, row * p.ldh + i, h);
    if constexpr (OUTK == NORM_16)
      store_out<H_OUT>(p.q, row * p.ldq + i, h * sc.rstd * w);
    else
      static_cast<uint8_t*>(p.q)[row * p.ldq + i] =
          sc.zero ? 0 : static_cast<uint8_t>(quant2<OUTK>(h * (w * part) * sc.qmul, 0.0f));
  }
  if (OUTK != NORM_16 && lane == 0) p.scales[row] = sc.scale;
}

// 8 elements of x and r to h, with their part of the row's sum and maxima.
template <bool BF16, int OUTK>
__device__ __forceinline__ void add_group(const uint4& xv, const uint4& rv, const uint4& wv,
                                          float (&h)[8], float& sum, uint2& mx) {
  const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
  const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
  const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = unpack2<BF16>(xw[j]), b = unpack2<BF16>(rw[j]), c = unpack2<BF16>(ww[j]);
    const float h0 = a.x + b.x, h1 = a.y + b.y;
    h[2 * j] = h0;
    h[2 * j + 1] = h1;
    sum += h0 * h0;
    sum += h1 * h1;
    if constexpr (OUTK != NORM_16) {
      mx.x = max(mx.x, max(abs_bits(h0 * c.x), abs_bits(h1 * c.y)));
      mx.y = max(mx.y, max(abs_bits(h0), abs_bits(h1)));
    }
  }
}

// Both outputs of 8 elements, group g of a row.
template <bool BF16, int OUTK>
__device__ __forceinline__ void store_group(const NormParams& p, int64_t row, int g, const float* v,
                                            const uint4& wv, const RowScale& sc) {
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h) + row * p.ldh)[g] =
      make_uint4(pack2<H_OUT>(v[0], v[1]), pack2<H_OUT>(v[2], v[3]), pack2<H_OUT>(v[4], v[5]),
                 pack2<H_OUT>(v[6], v[7]));
  const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 c = unpack2<BF16>(ww[j]);
    if constexpr (OUTK == NORM_16)
      o[j] = pack2<H_OUT>(v[2 * j] * sc.rstd * c.x, v[2 * j + 1] * sc.rstd * c.y);
    else
      o[j] = sc.zero ? 0u : quant2<OUTK>(v[2 * j] * c.x * sc.qmul, v[2 * j + 1] * c.y * sc.qmul);
  }
  if constexpr (OUTK == NORM_16)
    reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q) + row * p.ldq)[g] =
        make_uint4(o[0], o[1], o[2], o[3]);
  else
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.q) + row * p.ldq)[g] =
        make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// One row to a warp (four to a block of 128) or to a block, held in registers:
// PER groups of 8 elements a thread. Needs 16-byte aligned rows and cols a
// multiple of 8. The block of a wide row has just the threads that the row
// needs: with a fixed block, the idle part of it cost up to a third (8192 rows
// of 5000: 68 us).
template <bool BF16, int OUTK, bool WARP_ROW, int PER>
__global__ void __launch_bounds__(WARP_ROW || PER == 4 ? 128 : 1024) add_rms_norm_kernel(const NormParams p) {
  __shared__ float s_sum[32];
  __shared__ uint2 s_max[32];
  const int lanes = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
  const int lane = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)
                               : static_cast<int64_t>(blockIdx.x);
  const bool live = row < p.rows;
  const int groups = p.cols >> 3;
  grid_dependency_wait();
  uint4 xv[PER], rv[PER], wv[PER];
  const uint4* px = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.ldx);
  const uint4* pr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.r) + row * p.ldr);
  const uint4* pw = static_cast<const uint4*>(p.w);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = lane + i * lanes;
    const bool in = live && g < groups;
    xv[i] = in ? __ldcs(px + g) : make_uint4(0, 0, 0, 0);  // read once
    rv[i] = in ? __ldcs(pr + g) : make_uint4(0, 0, 0, 0);
    wv[i] = in ? pw[g] : make_uint4(0, 0, 0, 0);  // (coherent: the call before may have written it)
  }
  float h[PER][8];
  float sum = 0.0f;
  uint2 mx = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < PER; ++i) add_group<BF16, OUTK>(xv[i], rv[i], wv[i], h[i], sum, mx);
  row_reduce<WARP_ROW>(sum, mx, s_sum, s_max);
  grid_launch_dependents();
  if (!live) return;
  if (products_overflow<BF16, OUTK>(mx)) {
    finish_row<BF16, OUTK, WARP_ROW ? 32 : 0>(p, row, sum, mx, s_sum, s_max);
    return;
  }
  const RowScale sc = row_scale<OUTK>(sum, mx, p.cols, p.eps);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = lane + i * lanes;
    if (g < groups) store_group<BF16, OUTK>(p, row, g, h[i], wv[i], sc);
  }
  if (OUTK != NORM_16 && lane == 0) p.scales[row] = sc.scale;
}

// Many wide rows: a fixed number of blocks, each going through every
// gridDim.x-th row with a ring of rows ahead of it in shared memory, filled by
// bulk copies. The copies of the next rows run while a row is reduced and
// stored, whatever the block's size; w stays in registers. PER groups of 8
// elements a thread.
constexpr int NORM_MAX_STAGES = 4;
__host__ __device__ constexpr int norm_row_bytes(int cols) { return (2 * cols + 127) & ~127; }
__host__ __device__ constexpr int norm_ring_smem(int cols, int stages) {
  return stages * 2 * norm_row_bytes(cols) + 128;
}

template <bool BF16, int OUTK, int PER, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) add_rms_norm_ring_kernel(const NormParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float s_sum[2][32];
  __shared__ uint2 s_max[2][32];
  __shared__ __align__(8) uint64_t bars[NORM_MAX_STAGES];
  __shared__ int abort_word;
  const int S = p.stages;
  const int row_bytes = norm_row_bytes(p.cols);
  const uint32_t bytes = static_cast<uint32_t>(2 * p.cols);
  const int groups = p.cols >> 3;
  const uint32_t bar0 = smem_addr(bars), ring0 = smem_addr(ring);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  const WaitCtl ctl{p.timeout_ns, p.error_word, &abort_word};
  const uint64_t pol = policy_evict_first();  // read once
  auto fetch = [&](int64_t row, int s) {
    const uint32_t bar = bar0 + 8 * s, dst = ring0 + static_cast<uint32_t>(2 * s * row_bytes);
    mbar_arrive_expect_tx(bar, 2 * bytes);
    bulk_load_1d(dst, static_cast<const uint16_t*>(p.x) + row * p.ldx, bytes, bar, pol);
    bulk_load_1d(dst + row_bytes, static_cast<const uint16_t*>(p.r) + row * p.ldr, bytes, bar, pol);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + static_cast<int64_t>(s) * gridDim.x < p.rows && !(p.inject_stall && s == 1))
        fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  uint4 wv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = threadIdx.x + i * blockDim.x;
    wv[i] = g < groups ? static_cast<const uint4*>(p.w)[g] : make_uint4(0, 0, 0, 0);
  }
  int s = 0;
  uint32_t phase = 0, odd = 0;
  bool ok = true;      // this thread has seen every row so far arrive
  int64_t landed = 0;  // rows of this block that it has
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    // (a wait that runs out leaves this row and the block's next ones wrong and
    // says so; the loop and its barriers go on, without waits and copies)
    ok = ok && wait_bounded_lazy(bar0 + 8 * s, phase, ctl, WAIT_MMA_FULL);
    landed += ok;
    const uint4* sx = reinterpret_cast<const uint4*>(ring + 2 * s * row_bytes);
    const uint4* sr = reinterpret_cast<const uint4*>(ring + (2 * s + 1) * row_bytes);
    float h[PER][8];
    float sum = 0.0f;
    uint2 mx = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = threadIdx.x + i * blockDim.x;
      const uint4 none = make_uint4(0, 0, 0, 0);
      add_group<BF16, OUTK>(g < groups ? sx[g] : none, g < groups ? sr[g] : none, wv[i], h[i], sum, mx);
    }
    // (its barrier also says that the stage has been read; its buffers
    // alternate, so a fast warp's next row leaves a slow one's sums alone)
    row_reduce<false>(sum, mx, s_sum[odd], s_max[odd]);
    // (into a place whose last copy has landed, and into no other)
    const int64_t next = row + static_cast<int64_t>(S) * gridDim.x;
    if (threadIdx.x == 0 && ok && next < p.rows) fetch(next, s);
    if (products_overflow<BF16, OUTK>(mx)) {
      finish_row<BF16, OUTK, 0>(p, row, sum, mx, s_sum[odd], s_max[odd]);
    } else {
      const RowScale sc = row_scale<OUTK>(sum, mx, p.cols, p.eps);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int g = threadIdx.x + i * blockDim.x;
        if (g < groups) store_group<BF16, OUTK>(p, row, g, h[i], wv[i], sc);
      }
      if (OUTK != NORM_16 && threadIdx.x == 0) p.scales[row] = sc.scale;
    }
    odd ^= 1u;
    if (++s == S) {
      s = 0;
      phase ^= 1u;
    }
  }
  grid_launch_dependents();
  if (threadIdx.x == 0 && !ok) {
    // let the copies in flight land before the block exits: up to S rows past
    // those that have
    for (int64_t i = landed; i < landed + S && blockIdx.x + i * gridDim.x < p.rows; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar0 + 8 * static_cast<uint32_t>(i % S), static_cast<uint32_t>(i / S) & 1u) &&
             global_timer_ns() - t0 < ctl.timeout_ns) {
      }
    }
  }
}

// Rows of any width, alignment and pitch: one block to a row, element by
// element, x + r formed a second time for the outputs (the second read comes
// from L2).
template <bool BF16, int OUTK>
__global__ void __launch_bounds__(512) add_rms_norm_any_kernel(const NormParams p) {
  __shared__ float s_sum[32];
  __shared__ uint2 s_max[32];
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
  row_reduce<false>(sum, mx, s_sum, s_max);
  grid_launch_dependents();
  finish_row<BF16, OUTK, 512>(p, row, sum, mx, s_sum, s_max);
}

}  // namespace sptg
