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
// both given). 16384 rows of 4096 take 87 us (6.1 TB/s) and 149 us (5.4 TB/s; issue slots
// 60 % taken, and two exchanges between the warps to a row). A row stays on the SM between its
// reductions. Backwards a block
// goes through rows of its own choice and keeps two sums over rows for each column
// in registers: of dv hn, which is dw2, and of e = dh' yn, from which both dw1 = g e and a
// column's dg = w1 e follow (g inside the sum where it differs from row to row). They go
// to a workspace, and a second kernel adds those of all blocks up, in a fixed order.
#pragma once

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "shifted.cuh"

namespace sptg {

enum GateKind : int { GATE_NONE = 0, GATE_COLS = 1, GATE_ROWS = 2, GATE_FULL = 3 };

// A ring of rows in shared memory, filled by bulk copies that run ahead of the
// block: the rows of up to five operands and a barrier to a stage. Row i of a block
// is row blockIdx.x + i * gridDim.x of the call.
constexpr int GATE_MAX_STAGES = 4;
constexpr int GATE_MAX_OPS = 5;
// (A cut row, below, takes up to 62 bytes more.)
__host__ __device__ constexpr int gate_row_bytes(int cols, bool cut) { return (2 * cols + (cut ? 64 : 0) + 127) & ~127; }
__host__ __device__ constexpr int gate_ring_smem(int cols, int ops, int stages, bool cut) {
  return stages * ops * gate_row_bytes(cols, cut) + 128;
}

struct GateRing {
  const void* src[GATE_MAX_OPS];  // y, x, dh if given, dv if given, the gate if full
  int64_t ld[GATE_MAX_OPS];
  int ops, stages;
  unsigned int* error_word;  // where a wait that runs out reports
  uint64_t timeout_ns;
  int inject_stall;          // test hook: a block's second row is never copied
};

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
  GateRing ring;
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
  int parts;         // CTAs of a cluster that share a row (1: none do)
  int part_cols;     // columns of each, a multiple of 8 (the last: what is left)
  float* part;       // [2][blocks][cols]: sums of dv hn, and of e
};

struct ColumnSumParams {
  const float* part;
  int blocks, cols, out_kind;
  void* dw2;
  void* dw1;         // null: not wanted
  void* dgate;       // of columns, or null
  const void* w1;    // what the second sum is multiplied by for dgate (null: 1)
  const void* gate;  // and for dw1 (null: 1)
};

// Sums over a block, the same for each thread: lanes by halves, then warps in
// turn. s: a place for each warp's sums.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float4* s) {
  static_assert(N <= 4, "a warp's sums are one 16-byte word");
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = static_cast<int>(blockDim.x) >> 5;
  if ((threadIdx.x & 31) == 0)
    s[threadIdx.x >> 5] = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.0f, N > 2 ? v[N > 2 ? 2 : 0] : 0.0f,
                                      N > 3 ? v[N > 3 ? 3 : 0] : 0.0f);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    const float4 a = s[w];
    const float part[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += part[i];
  }
}

// Sums over a row, of a block or (WIDE) of a cluster whose CTAs share it: the blocks' sums go
// to all of them, and are added up by rank.
constexpr int GATE_MAX_PARTS = 8;
template <bool WIDE, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float4* s, float4* of_parts, int parts, int rank) {
  block_sums<N>(v, s);
  if constexpr (!WIDE) return;
  if (static_cast<int>(threadIdx.x) < parts) {
    const uint32_t to = map_to_cta(smem_addr(of_parts + rank), threadIdx.x);
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[0]), "f"(N > 1 ? v[N > 1 ? 1 : 0] : 0.0f),
                 "f"(N > 2 ? v[N > 2 ? 2 : 0] : 0.0f), "f"(0.0f)
                 : "memory");
  }
  __syncwarp();
  cluster_sync();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int r = 0; r < parts; ++r) {
    const float4 a = of_parts[r];
    const float part[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += part[i];
  }
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

// Two floats in one register pair and the instructions that take two at a time:
// the ring kernels are short of issue slots and registers, not of arithmetic.
typedef unsigned long long float_pair;
__device__ __forceinline__ float_pair pair_of(float a, float b) {
  float_pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float_pair pair_of(float a) { return pair_of(a, a); }
__device__ __forceinline__ float2 floats_of(float_pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ float_pair fma2(float_pair a, float_pair b, float_pair c) {
  float_pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float_pair mul2(float_pair a, float_pair b) {
  float_pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float_pair add2(float_pair a, float_pair b) {
  float_pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum_of(float_pair p) {
  const float2 f = floats_of(p);
  return f.x + f.y;
}

template <bool BF16>
__device__ __forceinline__ void pair_unpack(const uint4& v, float_pair (&f)[4]) {
  float a[8];
  gate_unpack<BF16>(v, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair_of(a[2 * i], a[2 * i + 1]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pair_pack(const float_pair (&f)[4]) {
  constexpr int OUT = BF16 ? OUT_BF16 : OUT_F16;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = floats_of(f[i]);
    w[i] = pack2<OUT>(a.x, a.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ const uint4* row_pieces(const void* p, int64_t row, int64_t ld) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row * ld);
}
__device__ __forceinline__ uint4* row_pieces(void* p, int64_t row, int64_t ld) {
  return reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row * ld);
}

// 1 / sqrt(sumsq * inv_cols + eps): the approximation and a step of Newton's. (An
// infinite sum: 0; the step would make it NaN. NaN stays.)
__device__ __forceinline__ float reciprocal_rms(float sumsq, float inv_cols, float eps) {
  const float m = fmaf(sumsq, inv_cols, eps), r = rsqrtf(m);
  return m == INFINITY ? 0.0f : r * fmaf(-0.5f * m * r, r, 1.5f);
}

// One row to a block, PER pieces of 8 elements a thread (not ALIGNED: pieces by h's
// 16-byte boundaries, so that h may be y or x). h may be y or x: each thread has read
// what it writes.
template <bool BF16, int PER, bool ALIGNED>
__global__ void __launch_bounds__(1024) gate_norm_kernel(const __grid_constant__ GateNormParams p) {
  __shared__ float4 s_sum[2][32];
  const int64_t row = blockIdx.x;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  const uint16_t* y = static_cast<const uint16_t*>(p.y) + row * p.ldy;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ldx;
  uint16_t* h_row = static_cast<uint16_t*>(p.h) + row * p.ldh;
  uint16_t* v_row = static_cast<uint16_t*>(p.v) + row * p.ldv;
  const uint16_t* w1 = static_cast<const uint16_t*>(p.w1);
  const uint16_t* w2 = static_cast<const uint16_t*>(p.w2);
  const bool by_column = p.gate_kind == GATE_COLS || p.gate_kind == GATE_FULL;
  const uint16_t* gate = static_cast<const uint16_t*>(p.gate) + (p.gate_kind == GATE_FULL ? row * p.ldg : 0);
  const int start = ALIGNED ? 0 : -shift_of(h_row);
  // Rows of dense tensors lie alike, and need no shifts (16384 rows of 4097: 156 us, with
  // shifts 193 us; a ring of such rows, in which fewer warps run, 230 us).
  const bool alike = shift_of(y) + start == 0 && shift_of(x) + start == 0;
  const auto first = [&](int i) { return start + 8 * static_cast<int>(threadIdx.x + i * blockDim.x); };
  const auto load = [&](const uint16_t* from, int i) {
    return first(i) < p.cols ? load_piece<ALIGNED>(from, first(i), p.cols) : none;
  };
  grid_dependency_wait();
  uint4 yv[PER], xv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if constexpr (ALIGNED) {  // read once
      yv[i] = first(i) < p.cols ? __ldcs(reinterpret_cast<const uint4*>(y + first(i))) : none;
      xv[i] = first(i) < p.cols ? __ldcs(reinterpret_cast<const uint4*>(x + first(i))) : none;
    }
  }
  uint4 w1v[PER], w2v[PER], gv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!ALIGNED) {
      if (inside_row(first(i), p.cols)) {
        if (alike) {
          yv[i] = *reinterpret_cast<const uint4*>(y + first(i));
          xv[i] = *reinterpret_cast<const uint4*>(x + first(i));
        } else {
          const ShiftedPiece a = load_words(y + first(i)), b = load_words(x + first(i));
          yv[i] = shifted(a);
          xv[i] = shifted(b);
        }
      } else {
        // (the row's ends: all loads in one branch, so that they are in flight together)
        const bool in = first(i) < p.cols;
        yv[i] = in ? load_elements(y, first(i), p.cols) : none;
        xv[i] = in ? load_elements(x, first(i), p.cols) : none;
        gv[i] = in && by_column ? load_elements(gate, first(i), p.cols) : none;
        w1v[i] = in && p.w1 ? load_elements(w1, first(i), p.cols) : none;
        w2v[i] = in ? load_elements(w2, first(i), p.cols) : none;
        continue;
      }
    }
    gv[i] = by_column ? load(gate, i) : none;
    w1v[i] = p.w1 ? load(w1, i) : none;
    w2v[i] = load(w2, i);
  }
  const float gr = p.gate_kind == GATE_ROWS ? gate_load<BF16>(p.gate, row * p.ldg) : 1.0f;
  float r1 = 1.0f;
  if (p.w1) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      float f[8];
      gate_unpack<BF16>(yv[i], f);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[0] += f[c] * f[c];
    }
    block_sums<1>(sum, s_sum[0]);
    r1 = reciprocal_rms(sum[0], inv_cols, p.eps);
  }
  float h[PER][8];
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float yf[8], xf[8], w[8], g[8];
    gate_unpack<BF16>(yv[i], yf);
    gate_unpack<BF16>(xv[i], xf);
    gate_unpack<BF16>(w1v[i], w);
    gate_unpack<BF16>(gv[i], g);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float u = p.w1 ? yf[c] * r1 * w[c] : yf[c];
      h[i][c] = p.alpha * xf[c] + (by_column ? g[c] : gr) * u;
      sum[0] += h[i][c] * h[i][c];
    }
  }
  block_sums<1>(sum, s_sum[1]);
  grid_launch_dependents();
  const float r2 = reciprocal_rms(sum[0], inv_cols, p.eps);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (first(i) >= p.cols) continue;
    float w[8];
    gate_unpack<BF16>(w2v[i], w);
    store_piece<ALIGNED>(h_row, first(i), p.cols, gate_pack<BF16>(h[i]));
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] *= h[i][c] * r2;
    store_piece<ALIGNED>(v_row, first(i), p.cols, gate_pack<BF16>(w));
  }
}

// Rows of any width: one to a block, element by element, read anew for each step
// (from L1 and L2; 1024 rows of 32768: 173 us, 1.6 TB/s). h may be y or x: each element is read for the
// last time by the thread that then writes it.
constexpr int GATE_ANY_THREADS = 512;

template <bool BF16>
__global__ void __launch_bounds__(GATE_ANY_THREADS) gate_norm_any_kernel(const __grid_constant__ GateNormParams p) {
  __shared__ float4 s_sum[2][32];
  constexpr int H_OUT = BF16 ? OUT_BF16 : OUT_F16;
  const int64_t row = blockIdx.x;
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
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
    r1 = reciprocal_rms(sum[0], inv_cols, p.eps);
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
  const float r2 = reciprocal_rms(sum[0], inv_cols, p.eps);
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

__device__ __forceinline__ const uint16_t* ring_src(const GateRing& r, int o, int64_t row) {
  return static_cast<const uint16_t*>(r.src[o]) + row * r.ld[o];
}

// Starts the copies of the block's row i into its stage (one thread). WIDE: of the
// columns from col0 on, by the clusters' numbers.
template <bool WIDE = false>
__device__ __forceinline__ void ring_fetch(const GateNormParams& p, int64_t i, int s, uint32_t bar0, uint32_t data0,
                                           uint64_t policy, unsigned group = 0, unsigned groups = 0, int col0 = 0,
                                           int part_cols = 0) {
  const int64_t row = WIDE ? group + i * groups : blockIdx.x + i * gridDim.x;
  if (row >= p.rows || (p.ring.inject_stall && i == 1)) return;
  const int cols = WIDE ? part_cols : p.cols;
  const uint32_t row_bytes = gate_row_bytes(cols, false), bytes = 2u * cols;
  uint32_t dst = data0 + s * p.ring.ops * row_bytes;
  mbar_arrive_expect_tx(bar0 + 8 * s, p.ring.ops * bytes);
#pragma unroll
  for (int o = 0; o < GATE_MAX_OPS; ++o)
    if (o < p.ring.ops) {
      bulk_load_1d(dst, ring_src(p.ring, o, row) + (WIDE ? col0 : 0), bytes, bar0 + 8 * s, policy);
      dst += row_bytes;
    }
}

// Rows cut by 16-byte boundaries, backwards. Bulk copies take whole 16-byte words, so they
// fetch the words that lie inside of a row, and 16 threads its first and last few
// elements, which lie in words that are other rows' too. In shared memory a row keeps its
// place between boundaries: element e of an operand whose rows start `shift` elements
// behind one is element 8 + shift + e of its buffer. What is before and behind the row
// there is zero, and stays so: blocks take rows a multiple of 8 apart, so
// that an operand's shift is the same for all rows of a block. Pieces are laid out by the
// rows that are written; an operand with another shift is read in two words. The pieces
// at a row's ends go through shared memory, from where 16 threads write an element each.
// (4096 rows of 5001 with a full gate: 165 us; with each row loaded into registers and its
// ends written element by element by the threads that hold them 262 us.)
struct RowCut {
  int head, words, tail;  // elements before the first whole word, words, elements behind
  __device__ __forceinline__ RowCut(int shift, int cols) {
    head = shift ? min(cols, 8 - shift) : 0;
    words = (cols - head) >> 3;
    tail = cols - head - 8 * words;
  }
  // The element that the i-th of 16 threads has, or -1: 8 before the words, 8 behind.
  __device__ __forceinline__ int end(int i, int cols) const {
    if (i < 8) return i < head ? i : -1;
    return i - 8 < tail ? cols - tail + i - 8 : -1;
  }
};

// One operand of a ring, or one element at the end of a row: where it is in the block's first
// row, how far apart the block's rows are, and where it goes.
struct RingPart {
  const uint16_t* at;  // null: none
  int64_t step;
  uint32_t bytes, offset;
};

constexpr int GATE_MAX_OUTS = 3;

// What the threads that move rows know. (In shared memory: registers are what the
// kernel is short of.)
struct RingCutShared {
  RingPart copies[GATE_MAX_OPS];
  RingPart in[16 * GATE_MAX_OPS];
  RingPart out[16 * GATE_MAX_OUTS];
  uint4 ends[2][GATE_MAX_OUTS][2];  // by the row's parity and output: first and last piece
  uint32_t bytes;                   // of a row, all operands
};
struct RingWholeShared {};

// Fills sh and the ring's zeros; the caller synchronises.
__device__ __forceinline__ void ring_setup(const GateNormParams& p, RingCutShared& sh, uint8_t* ring) {
  const int t = threadIdx.x, row_bytes = gate_row_bytes(p.cols, true);
  if (t < 32) {
    uint32_t bytes = 0;
    if (t < p.ring.ops) {
      const uint16_t* src = ring_src(p.ring, t, blockIdx.x);
      const RowCut cut(shift_of(src), p.cols);
      bytes = 16u * cut.words;
      sh.copies[t] = {src + cut.head, static_cast<int64_t>(gridDim.x) * p.ring.ld[t], bytes,
                      static_cast<uint32_t>(t * row_bytes + (cut.head ? 32 : 16))};
    }
    bytes = __reduce_add_sync(0xffffffffu, bytes);
    if (t == 0) sh.bytes = bytes;
  }
  if (t < 16 * p.ring.ops) {
    const int o = t >> 4;
    const uint16_t* src = ring_src(p.ring, o, blockIdx.x);
    const int shift = shift_of(src), e = RowCut(shift, p.cols).end(t & 15, p.cols);
    sh.in[t] = {e < 0 ? nullptr : src + e, static_cast<int64_t>(gridDim.x) * p.ring.ld[o], 2,
                static_cast<uint32_t>(o * row_bytes + 2 * (8 + shift + e))};
  }
  // zeros around the rows, in the words that no copy writes
  const uint4 none = make_uint4(0, 0, 0, 0);
  for (int i = t; i < p.ring.stages * p.ring.ops; i += blockDim.x) {
    const int shift = shift_of(ring_src(p.ring, i % p.ring.ops, blockIdx.x));
    uint4* w = reinterpret_cast<uint4*>(ring + i * row_bytes);
    const int last = 1 + ((shift + p.cols) >> 3);
    w[0] = none;
    if (shift) w[1] = none;
    w[last] = none;
    w[last + 1] = none;
  }
}

// An output's row ends: the threads' elements, where the pieces (that start `start`
// elements behind the row's first) are laid out by this output's boundaries. Returns
// whether they are.
__device__ __forceinline__ bool ring_output(const GateNormParams& p, RingCutShared& sh, int o, const void* out,
                                            int64_t ld, int start) {
  const uint16_t* row = static_cast<const uint16_t*>(out) + blockIdx.x * ld;
  const int shift = shift_of(row), i = static_cast<int>(threadIdx.x) - 16 * o;
  if (i >= 0 && i < 16) {
    const int e = shift + start == 0 ? RowCut(shift, p.cols).end(i, p.cols) : -1;
    sh.out[threadIdx.x] = {e < 0 ? nullptr : row + e, static_cast<int64_t>(gridDim.x) * ld, 2,
                           static_cast<uint32_t>(32 * o + (i < 8 ? 2 * (shift + i) : 16 + 2 * (i - 8)))};
  }
  return shift + start == 0;
}

// Starts the copies of the block's row i, of a cut row, into its stage (the first warp; a
// lane an operand).
__device__ __forceinline__ void ring_fetch_cut(const GateNormParams& p, const RingCutShared& sh, int64_t i, int s,
                                               uint32_t bar0, uint32_t data0, uint64_t policy) {
  if (blockIdx.x + i * gridDim.x >= p.rows || (p.ring.inject_stall && i == 1)) return;
  if (threadIdx.x == 0) mbar_arrive_expect_tx(bar0 + 8 * s, sh.bytes);
  __syncwarp();
  if (threadIdx.x < p.ring.ops) {
    const RingPart c = sh.copies[threadIdx.x];
    if (c.bytes > 0)
      bulk_load_1d(data0 + s * p.ring.ops * gate_row_bytes(p.cols, true) + c.offset, c.at + i * c.step, c.bytes,
                   bar0 + 8 * s, policy);
  }
}

// The first and last elements of row i, one a thread and operand: loaded when the row's
// copies are started, and stored a barrier later, so that nobody waits for them.
__device__ __forceinline__ void ends_load(const GateNormParams& p, const RingCutShared& sh, int64_t i, uint16_t& v) {
  if (threadIdx.x >= 16 * p.ring.ops || blockIdx.x + i * gridDim.x >= p.rows) return;
  const RingPart e = sh.in[threadIdx.x];
  if (e.at) v = e.at[i * e.step];
}
__device__ __forceinline__ void ends_store(const GateNormParams& p, const RingCutShared& sh, int64_t i, uint8_t* stage,
                                           uint16_t v) {
  if (threadIdx.x >= 16 * p.ring.ops || blockIdx.x + i * gridDim.x >= p.rows) return;
  const RingPart e = sh.in[threadIdx.x];
  if (e.at) *reinterpret_cast<uint16_t*>(stage + e.offset) = v;
}
// Those of the outputs, written behind the barrier that follows them.
__device__ __forceinline__ void ends_write(const RingCutShared& sh, int outs, int64_t i, int odd) {
  if (threadIdx.x >= 16 * outs) return;
  const RingPart e = sh.out[threadIdx.x];
  if (e.at)
    const_cast<uint16_t*>(e.at)[i * e.step] =
        *reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(sh.ends[odd]) + e.offset);
}

static __device__ __noinline__ void store_apart(uint16_t* row, int first, int cols, uint4 v) {
  store_shifted(row, first, cols, v);
}

// A piece of an output's cut row. alike: whether pieces are laid out by this output's boundaries.
__device__ __forceinline__ void ring_store(RingCutShared& sh, int o, int odd, bool alike, uint16_t* row, int first,
                                           int cols, const uint4& v) {
  if (alike && first >= 0 && first + 8 <= cols)
    *reinterpret_cast<uint4*>(row + first) = v;
  else if (alike)
    sh.ends[odd][o][first < 0 ? 0 : 1] = v;
  else
    store_apart(row, first, cols, v);
}

// Piece `at` of an operand in a ring, `apart` elements behind the pieces' own shift.
template <bool CUT>
__device__ __forceinline__ uint4 ring_piece(const uint8_t* row, int at, int apart) {
  const uint4* w = reinterpret_cast<const uint4*>(row) + at;
  if (!CUT) return w[0];
  w += 1 + (apart >> 3);
  if ((apart & 7) == 0) return w[0];
  return shifted(ShiftedPiece{w[0], w[1], apart & 7});
}

// Lets the copies in flight land before the block leaves: those up to a ring past
// the rows that have.
__device__ __forceinline__ void ring_drain(const GateNormParams& p, unsigned first, unsigned step, int64_t landed, uint32_t bar0) {
  for (int64_t i = landed; i < landed + p.ring.stages && first + i * step < p.rows; ++i) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar0 + 8 * static_cast<uint32_t>(i % p.ring.stages),
                          static_cast<uint32_t>(i / p.ring.stages) & 1u) &&
           global_timer_ns() - t0 < p.ring.timeout_ns) {
    }
  }
}

// Forwards, many rows: a fixed number of blocks with a ring each. PER pieces of 8
// elements a thread.
template <bool BF16, int PER>
__global__ void __launch_bounds__(512) gate_norm_ring_kernel(const __grid_constant__ GateNormParams p) {
  extern __shared__ __align__(128) uint8_t ring_data[];
  // (alternating, so that a fast warp's next row leaves a slow one's sums alone)
  __shared__ float4 s_sum[2][2][32];
  __shared__ __align__(8) uint64_t bars[GATE_MAX_STAGES];
  __shared__ int abort_word;
  const int pieces = p.cols >> 3;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const bool by_column = p.gate_kind == GATE_COLS || p.gate_kind == GATE_FULL;
  const bool full = p.gate_kind == GATE_FULL;
  const float inv_cols = 1.0f / static_cast<float>(p.cols);
  const uint32_t bar0 = smem_addr(bars), data0 = smem_addr(ring_data);
  const int row_bytes = gate_row_bytes(p.cols, false), stage_bytes = p.ring.ops * row_bytes;
  const uint64_t policy = policy_evict_first();  // read once
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring.stages; ++s) mbar_init(bar0 + 8 * s, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_dependency_wait();
  if (threadIdx.x == 0)
    for (int i = 0; i < p.ring.stages; ++i) ring_fetch(p, i, i, bar0, data0, policy);
  const WaitCtl ctl{p.ring.timeout_ns, p.ring.error_word, &abort_word};
  uint4 w1[PER], w2[PER], gv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool in = at < pieces;
    w1[i] = in && p.w1 ? static_cast<const uint4*>(p.w1)[at] : none;
    w2[i] = in ? static_cast<const uint4*>(p.w2)[at] : none;
    gv[i] = in && p.gate_kind == GATE_COLS ? static_cast<const uint4*>(p.gate)[at] : none;
  }
  const float_pair alpha = pair_of(p.alpha);
  // The sum of squares of y is formed a row ahead, so that it goes through the
  // threads together with the row's own: one barrier a row.
  const auto square_sum = [&](int stage) {
    const uint4* sy = reinterpret_cast<const uint4*>(ring_data + stage * stage_bytes);
    float_pair sq = pair_of(0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair y[4];
      pair_unpack<BF16>(sy[at], y);
#pragma unroll
      for (int c = 0; c < 4; ++c) sq = fma2(y[c], y[c], sq);
    }
    return sum_of(sq);
  };
  int odd = 0, s = 0;
  uint32_t phase = 0;
  // This thread has seen every row so far arrive. (A wait that runs out leaves its
  // row and the block's next ones wrong and says so; the loop and its barriers go
  // on, without waits and copies.)
  bool ok = wait_bounded_lazy(bar0, 0, ctl, WAIT_MMA_FULL);
  int64_t landed = ok;
  float next[1] = {p.w1 ? square_sum(0) : 0.0f};
  block_sums<1>(next, s_sum[1][1]);
  int64_t n = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++n, odd ^= 1) {
    const float gr = p.gate_kind == GATE_ROWS ? gate_load<BF16>(p.gate, row * p.ldg) : 1.0f;
    const uint4* sy = reinterpret_cast<const uint4*>(ring_data + s * stage_bytes);
    const uint4* sx = reinterpret_cast<const uint4*>(ring_data + s * stage_bytes + row_bytes);
    const uint4* sg = reinterpret_cast<const uint4*>(ring_data + s * stage_bytes + 2 * row_bytes);
    const float r1 = p.w1 ? reciprocal_rms(next[0], inv_cols, p.eps) : 1.0f;
    float_pair h[PER][4];
    float_pair sq = pair_of(0.0f);
    const float_pair factor = pair_of(by_column ? r1 : r1 * gr);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair x[4], w[4], g[4];
      pair_unpack<BF16>(sy[at], h[i]);
      pair_unpack<BF16>(sx[at], x);
      if (full) gv[i] = sg[at];
      pair_unpack<BF16>(w1[i], w);
      pair_unpack<BF16>(gv[i], g);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float_pair u = mul2(h[i][c], factor);
        if (p.w1) u = mul2(u, w[c]);
        if (by_column) u = mul2(u, g[c]);
        h[i][c] = fma2(alpha, x[c], u);
        sq = fma2(h[i][c], h[i][c], sq);
      }
    }
    const int later = s + 1 == p.ring.stages ? 0 : s + 1;
    const uint32_t later_phase = later == 0 ? phase ^ 1u : phase;
    float sums[2] = {sum_of(sq), 0.0f};
    if (row + gridDim.x < p.rows) {
      ok = ok && wait_bounded_lazy(bar0 + 8 * later, later_phase, ctl, WAIT_MMA_FULL);
      landed += ok;
      if (p.w1) sums[1] = square_sum(later);
    }
    block_sums<2>(sums, s_sum[odd][0]);
    next[0] = sums[1];
    // (the stage has been read; into a place whose last copy has landed, no other)
    if (threadIdx.x == 0 && ok) ring_fetch(p, n + p.ring.stages, s, bar0, data0, policy);
    const float_pair r2 = pair_of(reciprocal_rms(sums[0], inv_cols, p.eps));
    uint4* ph = row_pieces(p.h, row, p.ldh);
    uint4* pv = row_pieces(p.v, row, p.ldv);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair w[4];
      pair_unpack<BF16>(w2[i], w);
      ph[at] = pair_pack<BF16>(h[i]);
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = mul2(mul2(h[i][c], r2), w[c]);
      pv[at] = pair_pack<BF16>(w);
    }
    s = later;
    phase = later_phase;
  }
  grid_launch_dependents();
  if (threadIdx.x == 0 && !ok) ring_drain(p, blockIdx.x, gridDim.x, landed, bar0);
}

// Backwards: a fixed number of blocks, PER pieces of 8 elements a thread, whose sums
// over rows stay in registers. GRAD_CUT: rows off 16-byte boundaries. GRAD_WIDE: rows that
// one block cannot hold, shared by the CTAs of a cluster, each with a part of the columns.
enum GradForm { GRAD_WHOLE, GRAD_CUT, GRAD_WIDE };

template <bool BF16, int PER, int GATE, bool BLOCK, int FORM>
__global__ void __launch_bounds__(512) gate_norm_grad_kernel(const __grid_constant__ GateNormGradParams p) {
  constexpr bool CUT = FORM == GRAD_CUT, WIDE = FORM == GRAD_WIDE;
  extern __shared__ __align__(128) uint8_t ring_data[];
  // (alternating, so that a fast warp's next row leaves a slow one's sums alone)
  __shared__ float4 s_sum[2][3][32];
  __shared__ __align__(8) uint64_t bars[GATE_MAX_STAGES];
  __shared__ int abort_word;
  __shared__ typename std::conditional<CUT, RingCutShared, RingWholeShared>::type sh;
  const GateNormParams& f = p.f;
  __shared__ float4 s_parts[WIDE ? 2 : 1][3][WIDE ? GATE_MAX_PARTS : 1];
  const unsigned parts = WIDE ? p.parts : 1, rank = WIDE ? blockIdx.x % parts : 0;
  const unsigned group = WIDE ? blockIdx.x / parts : blockIdx.x, groups = WIDE ? gridDim.x / parts : gridDim.x;
  const int col0 = WIDE ? static_cast<int>(rank) * p.part_cols : 0, cols = WIDE ? min(p.part_cols, f.cols - col0) : f.cols;
  int start = CUT ? -shift_of(static_cast<const uint16_t*>(p.dx) + blockIdx.x * p.lddx) : 0;
  // (rows that fill the block to the last piece leave no room for one more: stores in parts)
  if (CUT && (cols - start + 7) >> 3 > PER * static_cast<int>(blockDim.x)) start = 0;
  const int pieces = (cols - start + 7) >> 3;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const float inv_cols = 1.0f / static_cast<float>(f.cols);
  const int op_dv = p.dh ? 3 : 2, op_gate = f.ring.ops - 1;
  const uint32_t bar0 = smem_addr(bars), data0 = smem_addr(ring_data);
  const int row_bytes = gate_row_bytes(cols, CUT), stage_bytes = f.ring.ops * row_bytes;
  const uint64_t policy = policy_evict_first();  // read once
  if (threadIdx.x == 0) {
    for (int s = 0; s < f.ring.stages; ++s) mbar_init(bar0 + 8 * s, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  const auto slot_of = [&](int op) { return op <= 2 ? op : op == 3 ? op_dv : op_gate; };
  int apart[GATE_MAX_OPS] = {0, 0, 0, 0, 0};
  bool dx_alike = true, dg_alike = true, dy_alike = true;
  if constexpr (CUT) {
    ring_setup(f, sh, ring_data);
#pragma unroll
    for (int o = 0; o < GATE_MAX_OPS; ++o) {
      const bool given = o < 2 || (o == 2 && p.dh) || (o == 3 && p.dv) || (o == 4 && GATE == GATE_FULL);
      if (given) apart[o] = shift_of(ring_src(f.ring, slot_of(o), blockIdx.x)) + start;
    }
    dx_alike = ring_output(f, sh, 0, p.dx, p.lddx, start);
    dy_alike = ring_output(f, sh, 1, p.dy, p.lddy, start);
    if (GATE == GATE_FULL) dg_alike = ring_output(f, sh, 2, p.dgate, p.lddg, start);
  }
  constexpr int OUTS = GATE == GATE_FULL ? 3 : 2;
  if constexpr (WIDE)
    cluster_sync();  // (all CTAs are there)
  else
    __syncthreads();
  grid_dependency_wait();
  uint16_t end = 0;
  if constexpr (!CUT) {
    if (threadIdx.x == 0)
      for (int i = 0; i < f.ring.stages; ++i) ring_fetch<WIDE>(f, i, i, bar0, data0, policy, group, groups, col0, cols);
  } else {
    if (threadIdx.x < 32)
      for (int i = 0; i < f.ring.stages; ++i) ring_fetch_cut(f, sh, i, i, bar0, data0, policy);
    for (int i = 0; i < f.ring.stages; ++i) {
      ends_load(f, sh, i, end);
      ends_store(f, sh, i, ring_data + i * stage_bytes, end);
    }
    __syncthreads();
  }
  const WaitCtl ctl{f.ring.timeout_ns, f.ring.error_word, &abort_word};
  // a column's factors: of u in h (w1, and the gate of columns), and w2
  float_pair gw[PER][4];
  uint4 w2[PER];
  float_pair sum_w2[PER][4], sum_e[PER][4];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool in = at < pieces;
    const auto column = [&](const void* w) {
      if constexpr (WIDE) return in ? static_cast<const uint4*>(w)[(col0 >> 3) + at] : none;
      return in ? load_piece<!CUT>(static_cast<const uint16_t*>(w), start + 8 * at, f.cols) : none;
    };
    w2[i] = column(f.w2);
    if (BLOCK) pair_unpack<BF16>(column(f.w1), gw[i]);
    float_pair g[4];
    if (GATE == GATE_COLS) pair_unpack<BF16>(column(f.gate), g);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!BLOCK) gw[i][c] = pair_of(1.0f);
      if (GATE == GATE_COLS) gw[i][c] = mul2(gw[i][c], g[c]);
      sum_w2[i][c] = sum_e[i][c] = pair_of(0.0f);
    }
  }
  const float_pair alpha = pair_of(f.alpha);
  // y's sum of squares is formed a row ahead, so that it goes through the threads
  // together with other sums: two barriers a row, not three.
  const auto square_sum = [&](int stage) {
    float_pair sq = pair_of(0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair y[4];
      pair_unpack<BF16>(ring_piece<CUT>(ring_data + stage * stage_bytes, at, apart[0]), y);
#pragma unroll
      for (int c = 0; c < 4; ++c) sq = fma2(y[c], y[c], sq);
    }
    return sum_of(sq);
  };
  int odd = 0, s = 0;
  uint32_t phase = 0;
  // This thread has seen every row so far arrive. (A wait that runs out leaves its
  // row and the block's next ones wrong and says so; the loop and its barriers go
  // on, without waits and copies.)
  bool ok = wait_bounded_lazy(bar0, 0, ctl, WAIT_MMA_FULL);
  int64_t landed = ok, n = 0;
  float s1[1] = {0.0f};
  if (BLOCK) {
    s1[0] = square_sum(0);
    row_sums<WIDE>(s1, s_sum[1][0], s_parts[WIDE][0], parts, rank);
  }
  for (int64_t row = group; row < f.rows; row += groups, ++n, odd ^= 1) {
    const float gr = GATE == GATE_ROWS ? gate_load<BF16>(f.gate, row * f.ldg) : 1.0f;
    const uint8_t* stage = ring_data + s * stage_bytes;
    const auto store = [&](int o, bool alike, void* to, int64_t ld, int at, const float_pair (&v)[4]) {
      if constexpr (CUT)
        ring_store(sh, o, odd, alike, static_cast<uint16_t*>(to) + row * ld, start + 8 * at, f.cols, pair_pack<BF16>(v));
      else
        row_pieces(to, row, ld)[(col0 >> 3) + at] = pair_pack<BF16>(v);
    };
    // piece i of y, x, dh, dv or the gate
    const auto operand = [&](int op, int i) {
      return ring_piece<CUT>(stage + slot_of(op) * row_bytes, threadIdx.x + i * blockDim.x, apart[op]);
    };
    uint4 yv[PER], gv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (threadIdx.x + i * blockDim.x >= pieces) continue;
      yv[i] = operand(0, i);
      if (GATE == GATE_FULL) gv[i] = operand(4, i);
    }
    const float r1 = BLOCK ? reciprocal_rms(s1[0], inv_cols, f.eps) : 1.0f;
    const float_pair gr1 = pair_of(gr * r1), r1p = pair_of(r1);
    float_pair h[PER][4];  // then dh'
    float_pair dot = pair_of(0.0f), sq = pair_of(0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (threadIdx.x + i * blockDim.x >= pieces) continue;
      float_pair y[4], x[4], g[4], dv[4], w[4];
      pair_unpack<BF16>(yv[i], y);
      pair_unpack<BF16>(operand(1, i), x);
      if (GATE == GATE_FULL) pair_unpack<BF16>(gv[i], g);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float_pair u = mul2(y[c], gr1);
        if (BLOCK || GATE == GATE_COLS) u = mul2(u, gw[i][c]);
        if (GATE == GATE_FULL) u = mul2(u, g[c]);
        h[i][c] = fma2(alpha, x[c], u);
        sq = fma2(h[i][c], h[i][c], sq);
      }
      if (p.dv) {
        pair_unpack<BF16>(operand(3, i), dv);
        pair_unpack<BF16>(w2[i], w);
#pragma unroll
        for (int c = 0; c < 4; ++c) dot = fma2(mul2(dv[c], w[c]), h[i][c], dot);
      }
    }
    float s2[2] = {sum_of(sq), sum_of(dot)};
    if constexpr (CUT) {  // (of the row fetched a row ago, into the stage before this one)
      if (n > 0) ends_store(f, sh, n - 1 + f.ring.stages, ring_data + (s == 0 ? f.ring.stages - 1 : s - 1) * stage_bytes, end);
    }
    row_sums<WIDE>(s2, s_sum[odd][1], s_parts[WIDE ? odd : 0][1], parts, rank);
    if constexpr (CUT) {
      if (n > 0) ends_write(sh, OUTS, n - 1, odd ^ 1);
    }
    const float r2 = reciprocal_rms(s2[0], inv_cols, f.eps);
    const float m2 = s2[1] * r2 * inv_cols;
    const float_pair r2p = pair_of(r2), back = pair_of(-(r2 * m2)), grp = pair_of(gr);
    dot = pair_of(0.0f);  // of e and gw
    float_pair row_dg = pair_of(0.0f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair y[4], g[4], dh[4], dg[4];
      pair_unpack<BF16>(yv[i], y);
      if (GATE == GATE_FULL) pair_unpack<BF16>(gv[i], g);
      if (p.dh) {
        pair_unpack<BF16>(operand(2, i), dh);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) dh[c] = pair_of(0.0f);
      }
      if (p.dv) {
        float_pair dv[4], w[4];
        pair_unpack<BF16>(operand(3, i), dv);
        pair_unpack<BF16>(w2[i], w);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float_pair hn = mul2(h[i][c], r2p);
          sum_w2[i][c] = fma2(dv[c], hn, sum_w2[i][c]);
          h[i][c] = fma2(hn, back, fma2(mul2(dv[c], w[c]), r2p, dh[c]));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) h[i][c] = dh[c];
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float_pair e = mul2(h[i][c], mul2(y[c], r1p));
        if (GATE == GATE_FULL) {
          dg[c] = mul2(e, gw[i][c]);
          e = mul2(e, g[c]);
        } else if (GATE == GATE_ROWS) {
          row_dg = fma2(e, gw[i][c], row_dg);
          e = mul2(e, grp);
        }
        sum_e[i][c] = add2(sum_e[i][c], e);
        dot = fma2(e, gw[i][c], dot);
        dh[c] = mul2(alpha, h[i][c]);
      }
      store(0, dx_alike, p.dx, p.lddx, at, dh);
      if (GATE == GATE_FULL) store(2, dg_alike, p.dgate, p.lddg, at, dg);
    }
    const int later = s + 1 == f.ring.stages ? 0 : s + 1;
    const uint32_t later_phase = later == 0 ? phase ^ 1u : phase;
    float s3[3] = {sum_of(dot), sum_of(row_dg), 0.0f};
    if (row + groups < f.rows) {
      ok = ok && wait_bounded_lazy(bar0 + 8 * later, later_phase, ctl, WAIT_MMA_FULL);
      landed += ok;
      if (BLOCK) s3[2] = square_sum(later);
    }
    row_sums<WIDE>(s3, s_sum[odd][2], s_parts[WIDE ? odd : 0][2], parts, rank);
    s1[0] = s3[2];
    // (the stage has been read; into a place whose last copy has landed, no other)
    if constexpr (!CUT) {
      if (threadIdx.x == 0 && ok) ring_fetch<WIDE>(f, n + f.ring.stages, s, bar0, data0, policy, group, groups, col0, cols);
    } else {
      if (threadIdx.x < 32 && __all_sync(0xffffffffu, ok)) ring_fetch_cut(f, sh, n + f.ring.stages, s, bar0, data0, policy);
      ends_load(f, sh, n + f.ring.stages, end);
    }
    if (GATE == GATE_ROWS && threadIdx.x == 0 && rank == 0) store_kind(p.dgate, row, s3[1], p.out_kind);
    const float_pair back1 = pair_of(-(s3[0] * inv_cols * r1 * r1));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (at >= pieces) continue;
      float_pair y[4], g[4];
      pair_unpack<BF16>(yv[i], y);
      if (GATE == GATE_FULL) pair_unpack<BF16>(gv[i], g);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float_pair d = mul2(h[i][c], gr1);
        if (BLOCK || GATE == GATE_COLS) d = mul2(d, gw[i][c]);
        if (GATE == GATE_FULL) d = mul2(d, g[c]);
        h[i][c] = BLOCK ? fma2(y[c], back1, d) : d;
      }
      store(1, dy_alike, p.dy, p.lddy, at, h[i]);
    }
    s = later;
    phase = later_phase;
  }
  grid_launch_dependents();
  if constexpr (CUT) {
    __syncthreads();
    ends_write(sh, OUTS, n - 1, odd ^ 1);
  }
  if (threadIdx.x == 0 && !ok) ring_drain(f, group, groups, landed, bar0);
  const int64_t plane = static_cast<int64_t>(groups) * f.cols;
  float* part = p.part + static_cast<int64_t>(group) * f.cols + col0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    if (at >= pieces) continue;
    const auto sums_out = [&](float* to, const float_pair (&pairs)[4]) {
      float v[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 a = floats_of(pairs[c]);
        v[2 * c] = a.x;
        v[2 * c + 1] = a.y;
      }
      if constexpr (!CUT) {
#pragma unroll
        for (int c = 0; c < 8; c += 4)
          *reinterpret_cast<float4*>(to + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (start + 8 * at + c >= 0 && start + 8 * at + c < f.cols) to[c] = v[c];
      }
    };
    sums_out(part + start + 8 * at, sum_w2[i]);
    if (BLOCK || GATE == GATE_COLS) sums_out(part + plane + start + 8 * at, sum_e[i]);
  }
}

// The same for rows of any width and alignment, element by element (0.7 TB/s). The block's
// sums over rows lie in the workspace, each written by one thread only.
template <bool BF16>
__global__ void __launch_bounds__(GATE_ANY_THREADS) gate_norm_grad_any_kernel(const __grid_constant__ GateNormGradParams p) {
  __shared__ float4 s_sum[2][3][32];
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
      r1 = reciprocal_rms(s[0], inv_cols, f.eps);
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
    const float r2 = reciprocal_rms(s2[0], inv_cols, f.eps);
    const float m2 = s2[1] * r2 * inv_cols;
    const auto d_at = [&](int c, float dv, float hn) {
      return (p.dh ? gate_load<BF16>(p.dh, row * p.lddh + c) : 0.0f) +
             r2 * (dv * gate_load<BF16>(f.w2, c) - hn * m2);
    };
    float s3[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < f.cols; c += GATE_ANY_THREADS) {
      const float hn = h_at(c) * r2, dv = dv_at(c), d = d_at(c, dv, hn);
      part[c] = (first ? 0.0f : part[c]) + dv * hn;
      const float dg = d * u_at(c);
      float e = d * gate_load<BF16>(y, c) * r1;
      s3[0] += dg * gate_at(c);
      s3[1] += dg;
      if (f.gate_kind == GATE_FULL) store_out<OUT>(p.dgate, row * p.lddg + c, dg);
      if (f.gate_kind != GATE_COLS) e *= gate_at(c);
      if (f.w1 || f.gate_kind == GATE_COLS) part[plane + c] = (first ? 0.0f : part[plane + c]) + e;
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
template <bool BF16, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) gate_norm_columns_kernel(const __grid_constant__ ColumnSumParams p) {
  __shared__ float s[WARPS][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  grid_dependency_wait();
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
    if (blockIdx.y == 0) {
      store_kind(p.dw2, c, sum, p.out_kind);
    } else {
      if (p.dw1) store_kind(p.dw1, c, p.gate ? sum * gate_load<BF16>(p.gate, c) : sum, p.out_kind);
      if (p.dgate) store_kind(p.dgate, c, p.w1 ? sum * gate_load<BF16>(p.w1, c) : sum, p.out_kind);
    }
  }
}

}  // namespace sptg
