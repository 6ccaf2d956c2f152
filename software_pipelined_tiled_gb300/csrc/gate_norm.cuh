// gate_norm.cuh -- the end of a block: norm of the block's output, gate, scaled
// residual, and the norm before the next block; with its gradients.
//
//   u = y * w1 / rms(y)             (without w1: u = y)        rms(a)^2 = mean(a^2) + eps
//   h = alpha x + g u               (g: none, a value a column, a row, or an element)
//   v = h * w2 / rms(h)
//
// and backwards, with p = 1 / rms(y), q = 1 / rms(h), yn = y p, hn = h q:
//
//   dh' = dh + q (dv w2 - hn mean(dv w2 hn)),   dw2 = sum over rows of dv hn
//   dx  = alpha dh',   dg = dh' u (added up over what g was broadcast to)
//   du  = dh' g,       dw1 = sum over rows of du yn
//   dy  = p (du w1 - yn mean(du w1 yn))         (without w1: dy = du)
//
// Everything between the loads and the stores is 32 bits; nothing is kept from the
// forward call, rows' statistics are cheaper formed anew than written and read.
//
// Memory-bound: 8 bytes an element forward, 12 backward (16-bit rows, dh and dv
// both given). A row stays in registers between its reductions. Backwards a block
// goes through rows of its own choice and keeps the sums over rows (dw1, dw2, dg of
// columns) in registers; its sums go to a workspace and a second kernel adds
// those of all blocks up, in a fixed order.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace sptg {

enum GateKind : int { GATE_NONE = 0, GATE_COLS = 1, GATE_ROWS = 2, GATE_FULL = 3 };

struct GateNormParams {
  const void* y;
  const void* x;
  const void* w1;    // or null
  const void* w2;
  const void* gate;  // COLS: cols; ROWS: rows, ldg apart; FULL: rows x cols
  int64_t ldy, ldx, ldg;
  void* h;
  void* v;
  int64_t ldh, ldv;
  int64_t rows;
  int cols, gate_kind;
  float alpha, eps;
};

struct GateNormGradParams {
  GateNormParams f;  // (h and v unused)
  const void* dh;    // or null
  const void* dv;    // or null
  int64_t lddh, lddv;
  void* dy;
  void* dx;
  int64_t lddy, lddx;
  void* dgate;       // ROWS, FULL
  int64_t lddg;
  int out_kind;      // of ROWS' dgate: OUT_F32 or the rows' type
  float* part;       // [3][blocks][cols]: w2, w1, gate
};

struct ColumnSumParams {
  const float* part;
  int blocks, cols, out_kind;
  void* out[3];      // null: not wanted
};

// Sums over a block, the same for each thread: lanes by halves, then warps in
// turn. s: 32 * N floats.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* s) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = static_cast<int>(blockDim.x) >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i * 32 + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += s[i * 32 + w];
}

template <bool BF16>
__device__ __forceinline__ void gate_unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 gate_pack(const float (&f)[8]) {
  constexpr int OUT = BF16 ? OUT_BF16 : OUT_F16;
  return make_uint4(pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]), pack2<OUT>(f[4], f[5]),
                    pack2<OUT>(f[6], f[7]));
}

template <bool BF16>
__device__ __forceinline__ float gate_load(const void* p, int64_t i) {
  if constexpr (BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else
    return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ const uint4* row_pieces(const void* p, int64_t row, int64_t ld) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row * ld);
}
__device__ __forceinline__ uint4* row_pieces(void* p, int64_t row, int64_t ld) {
  return reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row * ld);
}

__device__ __forceinline__ float reciprocal_rms(float sumsq, int cols, float eps) {
  return 1.0f / sqrtf(sumsq / static_cast<float>(cols) + eps);
}

// One row to a block, PER pieces of 8 elements a thread.
template <bool BF16, int PER>
__global__ void __launch_bounds__(1024) gate_norm_kernel(const GateNormParams p) {
  __shared__ float s_sum[2][32];
  const int64_t row = blockIdx.x;
  const int pieces = p.cols >> 3;
  const uint4 none = make_uint4(0, 0, 0, 0);
  grid_dependency_wait();
  uint4 yv[PER], xv[PER], w1[PER], w2[PER], gv[PER];
  const uint4* py = row_pieces(p.y, row, p.ldy);
  const uint4* px = row_pieces(p.x, row, p.ldx);
  const bool by_column = p.gate_kind == GATE_COLS || p.gate_kind == GATE_FULL;
  const uint4* pg = row_pieces(p.gate, p.gate_kind == GATE_FULL ? row : 0, p.ldg);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool in = at < pieces;
    yv[i] = in ? __ldcs(py + at) : none;
    xv[i] = in ? __ldcs(px + at) : none;
    gv[i] = in && by_column ? pg[at] : none;
    w1[i] = in && p.w1 ? static_cast<const uint4*>(p.w1)[at] : none;
    w2[i] = in ? static_cast<const uint4*>(p.w2)[at] : none;
  }
  const float gr = p.gate_kind == GATE_ROWS ? gate_load<BF16>(p.gate, row * p.ldg) : 1.0f;
  float r1 = 1.0f;
  if (p.w1) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float y[8];
      gate_unpack<BF16>(yv[i], y);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[0] += y[c] * y[c];
    }
    block_sums<1>(sum, s_sum[0]);
    r1 = reciprocal_rms(sum[0], p.cols, p.eps);
  }
  float h[PER][8];
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float y[8], x[8], w[8], g[8];
    gate_unpack<BF16>(yv[i], y);
    gate_unpack<BF16>(xv[i], x);
    gate_unpack<BF16>(w1[i], w);
    gate_unpack<BF16>(gv[i], g);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float u = p.w1 ? y[c] * r1 * w[c] : y[c];
      h[i][c] = p.alpha * x[c] + (by_column ? g[c] : gr) * u;
      sum[0] += h[i][c] * h[i][c];
    }
  }
  block_sums<1>(sum, s_sum[1]);
  grid_launch_dependents();
  const float r2 = reciprocal_rms(sum[0], p.cols, p.eps);
  uint4* ph = row_pieces(p.h, row, p.ldh);
  uint4* pv = row_pieces(p.v, row, p.ldv);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    if (at >= pieces) continue;
    float w[8];
    gate_unpack<BF16>(w2[i], w);
    ph[at] = gate_pack<BF16>(h[i]);
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] *= h[i][c] * r2;
    pv[at] = gate_pack<BF16>(w);
  }
}

// Rows of any width and alignment: one to a block, element by element, read anew
// for each step (from L1 and L2). h may be y or x: each element is read for the
// last time by the thread that then writes it.
constexpr int GATE_ANY_THREADS = 512;

template <bool BF16>
__global__ void __launch_bounds__(GATE_ANY_THREADS) gate_norm_any_kernel(const GateNormParams p) {
  __shared__ float s_sum[2][32];
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const uint16_t* y = static_cast<const uint16_t*>(p.y) + row * p.ldy;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx;
  const bool by_column = p.gate_kind == GATE_COLS || p.gate_kind == GATE_FULL;
  const int64_t g0 = p.gate_kind == GATE_FULL ? row * p.ldg : 0;
  const float gr = p.gate_kind == GATE_ROWS ? gate_load<BF16>(p.gate, row * p.ldg) : 1.0f;
  float r1 = 1.0f;
  if (p.w1) {
    float sum[1] = {0.0f};
    for (int c = threadIdx.x; c < p.cols; c += GATE_ANY_THREADS) {
      const float a = gate_load<BF16>(y, c);
      sum[0] += a * a;
    }
    block_sums<1>(sum, s_sum[0]);
    r1 = reciprocal_rms(sum[0], p.cols, p.eps);
  }
  const auto h_at = [&](int c) {
    const float a = gate_load<BF16>(y, c);
    const float u = p.w1 ? a * r1 * gate_load<BF16>(p.w1, c) : a;
    return p.alpha * gate_load<BF16>(x, c) + (by_column ? gate_load<BF16>(p.gate, g0 + c) : gr) * u;
  };
  float sum[1] = {0.0f};
  for (int c = threadIdx.x; c < p.cols; c += GATE_ANY_THREADS) {
    const float h = h_at(c);
    sum[0] += h * h;
  }
  block_sums<1>(sum, s_sum[1]);
  grid_launch_dependents();
  const float r2 = reciprocal_rms(sum[0], p.cols, p.eps);
  for (int c = threadIdx.x; c < p.cols; c += GATE_ANY_THREADS) {
    const float h = h_at(c);
    store_out<H_OUT>(p.h, row * p.ldh + c, h);
    store_out<H_OUT>(p.v, row * p.ldv + c, h * r2 * gate_load<BF16>(p.w2, c));
  }
}

__device__ __forceinline__ void store_kind(void* p, int64_t i, float v, int kind) {
  if (kind == OUT_F32)
    store_out<OUT_F32>(p, i, v);
  else if (kind == OUT_BF16)
    store_out<OUT_BF16>(p, i, v);
  else
    store_out<OUT_F16>(p, i, v);
}

// Backwards: every gridDim.x-th row to a block, PER pieces of 8 elements a thread.
template <bool BF16, int PER, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS) gate_norm_grad_kernel(const GateNormGradParams p) {
  // (alternating, so that a fast warp's next row leaves a slow one's sums alone)
  __shared__ float s_sum[2][3][64];
  const GateNormParams& f = p.f;
  const int pieces = f.cols >> 3;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const bool by_column = f.gate_kind == GATE_COLS || f.gate_kind == GATE_FULL;
  const float inv_cols = 1.0f / static_cast<float>(f.cols);
  grid_dependency_wait();
  uint4 w1[PER], w2[PER], gv[PER];
  float sum_w2[PER][8], sum_w1[PER][8], sum_g[PER][8];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool in = at < pieces;
    w1[i] = in && f.w1 ? static_cast<const uint4*>(f.w1)[at] : none;
    w2[i] = in ? static_cast<const uint4*>(f.w2)[at] : none;
    gv[i] = in && f.gate_kind == GATE_COLS ? static_cast<const uint4*>(f.gate)[at] : none;
#pragma unroll
    for (int c = 0; c < 8; ++c) sum_w2[i][c] = sum_w1[i][c] = sum_g[i][c] = 0.0f;
  }
  int odd = 0;
  for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x, odd ^= 1) {
    uint4 yv[PER], xv[PER], dhv[PER], dvv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      const bool in = at < pieces;
      yv[i] = in ? __ldcs(row_pieces(f.y, row, f.ldy) + at) : none;
      xv[i] = in ? __ldcs(row_pieces(f.x, row, f.ldx) + at) : none;
      dhv[i] = in && p.dh ? __ldcs(row_pieces(p.dh, row, p.lddh) + at) : none;
      dvv[i] = in && p.dv ? __ldcs(row_pieces(p.dv, row, p.lddv) + at) : none;
      if (f.gate_kind == GATE_FULL) gv[i] = in ? __ldcs(row_pieces(f.gate, row, f.ldg) + at) : none;
    }
    const float gr = f.gate_kind == GATE_ROWS ? gate_load<BF16>(f.gate, row * f.ldg) : 1.0f;
    float r1 = 1.0f;
    if (f.w1) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float y[8];
        gate_unpack<BF16>(yv[i], y);
#pragma unroll
        for (int c = 0; c < 8; ++c) s[0] += y[c] * y[c];
      }
      block_sums<1>(s, s_sum[odd][0]);
      r1 = reciprocal_rms(s[0], f.cols, f.eps);
    }
    float h[PER][8];  // then dh' g
    float s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float y[8], x[8], w[8], g[8], dv[8], ww[8];
      gate_unpack<BF16>(yv[i], y);
      gate_unpack<BF16>(xv[i], x);
      gate_unpack<BF16>(w1[i], w);
      gate_unpack<BF16>(gv[i], g);
      gate_unpack<BF16>(dvv[i], dv);
      gate_unpack<BF16>(w2[i], ww);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float u = f.w1 ? y[c] * r1 * w[c] : y[c];
        h[i][c] = f.alpha * x[c] + (by_column ? g[c] : gr) * u;
        s2[0] += h[i][c] * h[i][c];
        s2[1] += dv[c] * ww[c] * h[i][c];
      }
    }
    block_sums<2>(s2, s_sum[odd][1]);
    const float r2 = reciprocal_rms(s2[0], f.cols, f.eps);
    const float m2 = s2[1] * r2 * inv_cols;
    float s3[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      float y[8], w[8], g[8], dv[8], ww[8], dh[8], dx[8], dg[8];
      gate_unpack<BF16>(yv[i], y);
      gate_unpack<BF16>(w1[i], w);
      gate_unpack<BF16>(gv[i], g);
      gate_unpack<BF16>(dvv[i], dv);
      gate_unpack<BF16>(dhv[i], dh);
      gate_unpack<BF16>(w2[i], ww);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float hn = h[i][c] * r2;
        const float d = dh[c] + r2 * (dv[c] * ww[c] - hn * m2);
        sum_w2[i][c] += dv[c] * hn;
        dx[c] = f.alpha * d;
        const float yn = y[c] * r1;
        const float u = f.w1 ? yn * w[c] : y[c];
        dg[c] = d * u;
        s3[1] += dg[c];
        const float du = d * (by_column ? g[c] : gr);
        h[i][c] = du;
        sum_w1[i][c] += du * yn;
        s3[0] += du * w[c] * yn;
        if (f.gate_kind == GATE_COLS) sum_g[i][c] += dg[c];
      }
      if (at < pieces) {
        row_pieces(p.dx, row, p.lddx)[at] = gate_pack<BF16>(dx);
        if (f.gate_kind == GATE_FULL) row_pieces(p.dgate, row, p.lddg)[at] = gate_pack<BF16>(dg);
      }
    }
    if (f.w1 || f.gate_kind == GATE_ROWS) block_sums<2>(s3, s_sum[odd][2]);
    if (f.gate_kind == GATE_ROWS && threadIdx.x == 0) store_kind(p.dgate, row, s3[1], p.out_kind);
    const float m1 = s3[0] * inv_cols;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float y[8], w[8], dy[8];
      gate_unpack<BF16>(yv[i], y);
      gate_unpack<BF16>(w1[i], w);
#pragma unroll
      for (int c = 0; c < 8; ++c) dy[c] = f.w1 ? r1 * (h[i][c] * w[c] - y[c] * r1 * m1) : h[i][c];
      row_pieces(p.dy, row, p.lddy)[at] = gate_pack<BF16>(dy);
    }
  }
  grid_launch_dependents();
  const int64_t plane = static_cast<int64_t>(gridDim.x) * f.cols;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * f.cols;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    if (at >= pieces) continue;
#pragma unroll
    for (int c = 0; c < 8; c += 4) {
      const int64_t to = at * 8 + c;
      *reinterpret_cast<float4*>(part + to) =
          make_float4(sum_w2[i][c], sum_w2[i][c + 1], sum_w2[i][c + 2], sum_w2[i][c + 3]);
      if (f.w1)
        *reinterpret_cast<float4*>(part + plane + to) =
            make_float4(sum_w1[i][c], sum_w1[i][c + 1], sum_w1[i][c + 2], sum_w1[i][c + 3]);
      if (f.gate_kind == GATE_COLS)
        *reinterpret_cast<float4*>(part + 2 * plane + to) =
            make_float4(sum_g[i][c], sum_g[i][c + 1], sum_g[i][c + 2], sum_g[i][c + 3]);
    }
  }
}

// The same for rows of any width and alignment, element by element. The block's
// sums over rows lie in the workspace, each written by one thread only.
template <bool BF16>
__global__ void __launch_bounds__(GATE_ANY_THREADS) gate_norm_grad_any_kernel(const GateNormGradParams p) {
  __shared__ float s_sum[2][3][64];
  constexpr int OUT = BF16 ? OUT_BF16 : OUT_F16;
  const GateNormParams& f = p.f;
  const bool by_column = f.gate_kind == GATE_COLS || f.gate_kind == GATE_FULL;
  const float inv_cols = 1.0f / static_cast<float>(f.cols);
  const int64_t plane = static_cast<int64_t>(gridDim.x) * f.cols;
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * f.cols;
  grid_dependency_wait();
  int odd = 0;
  for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x, odd ^= 1) {
    const bool first = row == blockIdx.x;
    const uint16_t* y = static_cast<const uint16_t*>(f.y) + row * f.ldy;
    const uint16_t* x = static_cast<const uint16_t*>(f.x) + row * f.ldx;
    const int64_t g0 = f.gate_kind == GATE_FULL ? row * f.ldg : 0;
    const float gr = f.gate_kind == GATE_ROWS ? gate_load<BF16>(f.gate, row * f.ldg) : 1.0f;
    float r1 = 1.0f;
    if (f.w1) {
      float s[1] = {0.0f};
      for (int c = threadIdx.x; c < f.cols; c += GATE_ANY_THREADS) {
        const float a = gate_load<BF16>(y, c);
        s[0] += a * a;
      }
      block_sums<1>(s, s_sum[odd][0]);
      r1 = reciprocal_rms(s[0], f.cols, f.eps);
    }
    const auto gate_at = [&](int c) { return by_column ? gate_load<BF16>(f.gate, g0 + c) : gr; };
    const auto u_at = [&](int c) {
      const float a = gate_load<BF16>(y, c);
      return f.w1 ? a * r1 * gate_load<BF16>(f.w1, c) : a;
    };
    const auto h_at = [&](int c) { return f.alpha * gate_load<BF16>(x, c) + gate_at(c) * u_at(c); };
    const auto dv_at = [&](int c) { return p.dv ? gate_load<BF16>(p.dv, row * p.lddv + c) : 0.0f; };
    float s2[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < f.cols; c += GATE_ANY_THREADS) {
      const float h = h_at(c);
      s2[0] += h * h;
      s2[1] += dv_at(c) * gate_load<BF16>(f.w2, c) * h;
    }
    block_sums<2>(s2, s_sum[odd][1]);
    const float r2 = reciprocal_rms(s2[0], f.cols, f.eps);
    const float m2 = s2[1] * r2 * inv_cols;
    const auto d_at = [&](int c, float dv, float hn) {
      return (p.dh ? gate_load<BF16>(p.dh, row * p.lddh + c) : 0.0f) +
             r2 * (dv * gate_load<BF16>(f.w2, c) - hn * m2);
    };
    float s3[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < f.cols; c += GATE_ANY_THREADS) {
      const float hn = h_at(c) * r2, dv = dv_at(c), d = d_at(c, dv, hn);
      part[c] = (first ? 0.0f : part[c]) + dv * hn;
      const float u = u_at(c), yn = gate_load<BF16>(y, c) * r1, dg = d * u, du = d * gate_at(c);
      s3[1] += dg;
      if (f.gate_kind == GATE_FULL) store_out<OUT>(p.dgate, row * p.lddg + c, dg);
      if (f.gate_kind == GATE_COLS) part[2 * plane + c] = (first ? 0.0f : part[2 * plane + c]) + dg;
      if (f.w1) {
        part[plane + c] = (first ? 0.0f : part[plane + c]) + du * yn;
        s3[0] += du * gate_load<BF16>(f.w1, c) * yn;
      }
    }
    if (f.w1 || f.gate_kind == GATE_ROWS) block_sums<2>(s3, s_sum[odd][2]);
    if (f.gate_kind == GATE_ROWS && threadIdx.x == 0) store_kind(p.dgate, row, s3[1], p.out_kind);
    const float m1 = s3[0] * inv_cols;
    for (int c = threadIdx.x; c < f.cols; c += GATE_ANY_THREADS) {
      const float d = d_at(c, dv_at(c), h_at(c) * r2), du = d * gate_at(c);
      store_out<OUT>(p.dx, row * p.lddx + c, f.alpha * d);
      store_out<OUT>(p.dy, row * p.lddy + c,
                     f.w1 ? r1 * (du * gate_load<BF16>(f.w1, c) - gate_load<BF16>(y, c) * r1 * m1) : du);
    }
  }
  grid_launch_dependents();
}

// The blocks' sums of 32 columns added up by a block: every 32nd block's to a
// warp, then the warps' in turn.
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) gate_norm_columns_kernel(const ColumnSumParams p) {
  __shared__ float s[WARPS][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  void* out = p.out[blockIdx.y];
  grid_dependency_wait();
  if (out == nullptr) return;
  const float* part = p.part + static_cast<int64_t>(blockIdx.y) * p.blocks * p.cols;
  float sum = 0.0f;
  if (c < p.cols) {
#pragma unroll 4
    for (int b = warp; b < p.blocks; b += WARPS) sum += part[static_cast<int64_t>(b) * p.cols + c];
  }
  s[warp][lane] = sum;
  __syncthreads();
  grid_launch_dependents();
  if (warp == 0 && c < p.cols) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += s[w][lane];
    store_kind(out, c, sum, p.out_kind);
  }
}

}  // namespace sptg
