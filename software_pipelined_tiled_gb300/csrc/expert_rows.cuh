// expert_rows.cuh -- rows on their way to the experts and back.
//
//   dispatch   place[t, j] = rank of entry t * top + j among all entries in the
//              order of their experts (entries of one expert in their own order;
//              those of no expert last),   sorted[place[t, j]] = x[t]
//   sum        out[t] = base[t] + sum_j w[t, j] y[place[t, j]]
//              (the combination of the experts' outputs; without w and base the
//              gradient of dispatch by x)
//   its gradients   dy[place[t, j]] = w[t, j] dout[t],   dw[t, j] = <y[place[t, j]], dout[t]>
//
// All but the sort are bound by memory: each row is read once and written once
// (16384 rows of 4096 to 8 places and back: 186, 181 and 333 us, 6.5 to 6.9 TB/s),
// and `place` is a permutation, so that each row has one writer and nothing needs
// an atomic. Rows go through registers in pieces of 8 elements (16 bytes), shifted
// together where width, pitch or address put them off 16-byte boundaries.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "shifted.cuh"

namespace sptg {

constexpr int DISPATCH_MAX_EXPERTS = 1024;
constexpr int SORT_WARPS = 32;
constexpr int SORT_MAX_CLUSTER = 16;
constexpr int SORT_STEPS = 4;  // of 32 entries, whose loads are in flight together

struct SortParams {
  const int32_t* experts;  // entries
  int32_t* places;
  int32_t* offsets;        // E + 1
  int64_t entries;
  int64_t per_warp;        // entries of a warp, a multiple of 32
  int E;
  int bits;                // of E
};

// Counts by warp and expert, then the totals of the CTA.
__host__ __device__ constexpr int sort_smem(int E) { return (SORT_WARPS + 1) * (E + 1) * 4; }

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Stable sort of the entries by expert, by counting: one cluster of CTAs, no
// atomics. Every warp has a run of neighbouring entries of its own. It takes 32 at
// a time, the lanes of equal experts find each other by the bits of their numbers,
// and it notes for each entry how many of its expert came before it in the run
// (in places). When all have been counted, a warp's entries of an expert start
// behind those of the warps and CTAs before it. (131072 entries: 12.2 us, 32768: 7.6 us;
// matching lanes by whole numbers instead of bits 52 us.)
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
    dispatch_sort_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ uint32_t counts[];  // [WARPS][bins], then the CTA's totals
  __shared__ uint32_t s_warp[WARPS];
  constexpr int THREADS = 32 * WARPS;
  constexpr uint32_t ALL = 0xffffffffu;
  const int bins = p.E + 1;  // (the last: entries of no expert)
  uint32_t* totals = counts + WARPS * bins;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t before_me = (1u << lane) - 1u;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
  for (int i = threadIdx.x; i < WARPS * bins; i += THREADS) counts[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  uint32_t* mine = counts + warp * bins;
  const int64_t begin = (static_cast<int64_t>(rank) * WARPS + warp) * p.per_warp;
  const int64_t end = min(p.entries, begin + p.per_warp);
  const auto bin_of = [&](int e) { return e < 0 || e >= p.E ? p.E : e; };
  for (int64_t i0 = begin; i0 < end; i0 += 32 * SORT_STEPS) {
    int b[SORT_STEPS];
#pragma unroll
    for (int k = 0; k < SORT_STEPS; ++k) {
      const int64_t i = i0 + 32 * k + lane;
      b[k] = i < end ? bin_of(p.experts[i]) : 0;
    }
#pragma unroll
    for (int k = 0; k < SORT_STEPS; ++k) {
      const int64_t i = i0 + 32 * k + lane;
      if (i - lane >= end) break;
      uint32_t same = __ballot_sync(ALL, i < end);
      for (int bit = 0; bit < p.bits; ++bit) {
        const bool one = (b[k] >> bit) & 1;
        const uint32_t ones = __ballot_sync(ALL, one);
        same &= one ? ones : ~ones;
      }
      const uint32_t n = i < end ? mine[b[k]] : 0u;
      __syncwarp();
      if (i < end) {
        p.places[i] = static_cast<int32_t>(n + __popc(same & before_me));
        if ((same & before_me) == 0) mine[b[k]] = n + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // entries of each expert in the warps before, and in the CTA
  for (int b = threadIdx.x; b < bins; b += THREADS) {
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) {
      const uint32_t n = counts[w * bins + b];
      counts[w * bins + b] = sum;
      sum += n;
    }
    totals[b] = sum;
  }
  cluster_sync();
  // this thread's expert: entries of it in the CTAs before this one, and in all
  const int e = threadIdx.x;
  uint32_t before = 0, all = 0;
  {
    const uint32_t at = smem_addr(totals + min(e, p.E));
    uint32_t n[SORT_MAX_CLUSTER];
#pragma unroll
    for (int c = 0; c < SORT_MAX_CLUSTER; ++c)
      n[c] = e < p.E && c < ctas ? ld_cluster_u32(map_to_cta(at, c)) : 0;
#pragma unroll
    for (int c = 0; c < SORT_MAX_CLUSTER; ++c) {
      if (c < rank) before += n[c];
      all += n[c];
    }
  }
  // entries of no expert in the CTAs before this one, the same for each warp
  uint32_t none_before = lane < rank ? ld_cluster_u32(map_to_cta(smem_addr(totals + p.E), lane)) : 0;
  none_before = __reduce_add_sync(ALL, none_before);
  // where each expert starts
  uint32_t sum = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(ALL, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  uint32_t base = 0, live = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const uint32_t n = s_warp[w];
    if (w < warp) base += n;
    live += n;
  }
  const uint32_t start = base + sum - all;
  if (rank == 0) {
    if (e < p.E) p.offsets[e] = static_cast<int32_t>(start);
    if (e == 0) p.offsets[p.E] = static_cast<int32_t>(live);
  }
  if (e < p.E) {
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) counts[w * bins + e] += start + before;
  }
  if (e < WARPS) counts[e * bins + p.E] += live + none_before;
  cluster_sync();  // (the totals have been read, and this CTA's counts are first places now)
  grid_launch_dependents();
#pragma unroll 4
  for (int64_t i = begin + lane; i < end; i += 32)
    p.places[i] += static_cast<int32_t>(mine[bin_of(p.experts[i])]);
}

struct RowsParams {
  const void* x;          // copy: x; sum, gradients: y
  int64_t ldx;
  int64_t x_rows;         // sum, gradients: rows of y
  const int32_t* places;  // rows x top
  const float* weights;   // rows x top, or null (1)
  const void* base;       // sum: or null
  int64_t ldb;
  const void* dout;       // gradients
  int64_t ldd;
  void* out;              // copy: sorted rows; sum: out; gradients: dy
  int64_t ldo;
  int64_t out_rows;       // copy: rows of out
  float* dweights;        // gradients: or null
  int cols, top;
  int64_t entries;        // gradients: of places, where blocks are there for the rows of dy
  int zero_blocks;        // that none of them names: how many, the first of the grid (0: such rows
  int zero_window;        // are left), and the rows that one looks at, a multiple of 32
};

constexpr int ROWS_THREADS = 128;
constexpr int ROWS_AT_ONCE = 8;  // entries of a row whose loads are in flight together

__device__ __forceinline__ const uint16_t* row_of(const void* base, int64_t row, int64_t ld) {
  return static_cast<const uint16_t*>(base) + row * ld;
}
__device__ __forceinline__ uint16_t* row_of(void* base, int64_t row, int64_t ld) {
  return static_cast<uint16_t*>(base) + row * ld;
}

template <bool BF16>
__device__ __forceinline__ void unpack_piece(const uint4& v, float (&f)[8]) {
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
__device__ __forceinline__ uint4 pack_piece(const float (&f)[8]) {
  constexpr int OUT = BF16 ? OUT_BF16 : OUT_F16;
  return make_uint4(pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]), pack2<OUT>(f[4], f[5]),
                    pack2<OUT>(f[6], f[7]));
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t v) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else
    return __half2float(__ushort_as_half(v));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_float(float v) {
  return static_cast<uint16_t>(pack2<BF16 ? OUT_BF16 : OUT_F16>(v, 0.0f));
}

// One thread's part of a row of x to the rows of out that `place(j)` names.
template <bool ALIGNED, typename Place>
__device__ __forceinline__ void copy_row(const RowsParams& p, int64_t row, Place place) {
  const uint16_t* x = row_of(p.x, row, p.ldx);
  const int thread = blockIdx.y * ROWS_THREADS + threadIdx.x, threads = gridDim.y * ROWS_THREADS;
  if constexpr (ALIGNED) {
    for (int c = 8 * thread; c < p.cols; c += 8 * threads) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + c);
      for (int j = 0; j < p.top; ++j) {
        const int64_t to = place(j);
        if (to >= 0 && to < p.out_rows) *reinterpret_cast<uint4*>(row_of(p.out, to, p.ldo) + c) = v;
      }
    }
  } else {  // cut by each row written; x from L1 for all but the first
    for (int j = 0; j < p.top; ++j) {
      const int64_t to = place(j);
      if (to < 0 || to >= p.out_rows) continue;
      uint16_t* out = row_of(p.out, to, p.ldo);
      const CutRow cut(out, p.cols);
#pragma unroll 2
      for (int c = cut.body + 8 * thread; c < cut.tail; c += 8 * threads)
        *reinterpret_cast<uint4*>(out + c) = shifted(load_words(x + c));
      for (int i = thread; i < cut.ends; i += threads) out[cut.end(i)] = x[cut.end(i)];
    }
  }
}

// Rows of x to their places: a block to a row and a part of its columns
// (blockIdx.y). A place outside of the sorted rows is passed over.
template <bool ALIGNED>
__global__ void __launch_bounds__(ROWS_THREADS) dispatch_copy_kernel(const __grid_constant__ RowsParams p) {
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const int32_t* places = p.places + row * p.top;
  copy_row<ALIGNED>(p, row, [&](int j) { return places[j]; });
  grid_launch_dependents();
}

// Few entries, in one launch: every block finds the places of its own row by
// counting the entries that go before each of them, and copies the row; one more
// block (the last) counts the experts' entries for the offsets. (4096 entries of 4096
// columns: 14.1 us, sorted first 15.5; 2048: 7.3 and 10.4; the work goes with the
// square: 8192 entries sorted 20.6.)
constexpr int SMALL_ENTRIES = 4096;

template <bool ALIGNED>
__global__ void __launch_bounds__(ROWS_THREADS)
    dispatch_small_kernel(const __grid_constant__ RowsParams p, const __grid_constant__ SortParams s) {
  __shared__ int s_count[DISPATCH_MAX_EXPERTS + 1];
  __shared__ int s_place[SMALL_ENTRIES];
  constexpr uint32_t ALL = 0xffffffffu;
  const int n = static_cast<int>(s.entries), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto bin_at = [&](int i) {
    const int e = s.experts[i];
    return e < 0 || e >= s.E ? s.E : e;
  };
  grid_dependency_wait();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y != 0) return;
    for (int e = threadIdx.x; e <= s.E; e += ROWS_THREADS) s_count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += ROWS_THREADS) atomicAdd(&s_count[bin_at(i)], 1);
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int e0 = 0; e0 <= s.E; e0 += 32) {
        const int mine = e0 + lane < s.E ? s_count[e0 + lane] : 0;
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(ALL, sum, o);
          if (lane >= o) sum += up;
        }
        if (e0 + lane <= s.E) s.offsets[e0 + lane] = base + sum - mine;
        base += __shfl_sync(ALL, sum, 31);
      }
    }
    return;
  }
  const int64_t row = blockIdx.x;
  const int first = static_cast<int>(row) * p.top;
  for (int j = threadIdx.x; j < p.top; j += ROWS_THREADS) s_place[j] = 0;
  __syncthreads();
  // every fourth run of 32 entries to a warp, against eight of the row's at a time
  for (int j0 = 0; j0 < p.top; j0 += ROWS_AT_ONCE) {
    int mine[ROWS_AT_ONCE], before[ROWS_AT_ONCE];
#pragma unroll
    for (int j = 0; j < ROWS_AT_ONCE; ++j) {
      mine[j] = j0 + j < p.top ? bin_at(first + j0 + j) : -1;
      before[j] = 0;
    }
    for (int i = threadIdx.x; i < n; i += ROWS_THREADS) {
      const int b = bin_at(i);
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j)
        before[j] += b < mine[j] || (b == mine[j] && i < first + j0 + j);
    }
#pragma unroll
    for (int j = 0; j < ROWS_AT_ONCE; ++j) {
      const int sum = __reduce_add_sync(ALL, before[j]);
      if (lane == 0 && j0 + j < p.top) atomicAdd(&s_place[j0 + j], sum);
    }
  }
  __syncthreads();
  if (blockIdx.y == 0)
    for (int j = threadIdx.x; j < p.top; j += ROWS_THREADS) s.places[first + j] = s_place[j];
  copy_row<ALIGNED>(p, row, [&](int j) { return s_place[j]; });
  grid_launch_dependents();
}

// Sums of the rows that a row's places name, in 32 bits and in the order of the
// places, rounded once. A place outside of y counts as a row of zeros.
template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(ROWS_THREADS) combine_rows_kernel(const __grid_constant__ RowsParams p) {
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const int32_t* places = p.places + row * p.top;
  const float* weights = p.weights ? p.weights + row * p.top : nullptr;
  const uint16_t* base = p.base ? row_of(p.base, row, p.ldb) : nullptr;
  uint16_t* out = row_of(p.out, row, p.ldo);
  const int thread = blockIdx.y * ROWS_THREADS + threadIdx.x, threads = gridDim.y * ROWS_THREADS;
  // All rows' loads of a piece (Raw) are in flight before the first is used.
  const auto add_rows = [&](auto raw, auto load, auto add) {
    using Raw = decltype(raw);
    constexpr int AT_ONCE = ALIGNED ? ROWS_AT_ONCE : ROWS_AT_ONCE / 2;
    for (int j0 = 0; j0 < p.top; j0 += AT_ONCE) {
      Raw v[AT_ONCE];
      float w[AT_ONCE];
      bool in[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const int64_t from = j0 + j < p.top ? places[j0 + j] : -1;
        in[j] = from >= 0 && from < p.x_rows;
        w[j] = in[j] && weights ? weights[j0 + j] : 1.0f;
        if (in[j]) v[j] = load(row_of(p.x, from, p.ldx));
      }
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        if (in[j]) add(v[j], w[j]);
    }
  };
  float sum[8];
  const auto add_piece = [&](const uint4& v, float w) {
    float f[8];
    unpack_piece<BF16>(v, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += w * f[k];
  };
  const auto start_piece = [&](int c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
    if (base)
      unpack_piece<BF16>(ALIGNED ? *reinterpret_cast<const uint4*>(base + c) : shifted(load_words(base + c)), sum);
  };
  if constexpr (ALIGNED) {
    for (int c = 8 * thread; c < p.cols; c += 8 * threads) {
      start_piece(c);
      add_rows(uint4(), [&](const uint16_t* y) { return *reinterpret_cast<const uint4*>(y + c); }, add_piece);
      *reinterpret_cast<uint4*>(out + c) = pack_piece<BF16>(sum);
    }
  } else {
    const CutRow cut(out, p.cols);
    for (int c = cut.body + 8 * thread; c < cut.tail; c += 8 * threads) {
      start_piece(c);
      add_rows(ShiftedPiece(), [&](const uint16_t* y) { return load_words(y + c); },
               [&](const ShiftedPiece& v, float w) { add_piece(shifted(v), w); });
      *reinterpret_cast<uint4*>(out + c) = pack_piece<BF16>(sum);
    }
    for (int i = thread; i < cut.ends; i += threads) {
      const int c = cut.end(i);
      float s = base ? to_float<BF16>(base[c]) : 0.0f;
      add_rows(uint16_t(), [&](const uint16_t* y) { return y[c]; },
               [&](uint16_t v, float w) { s += w * to_float<BF16>(v); });
      out[c] = from_float<BF16>(s);
    }
  }
  grid_launch_dependents();
}

// Zeros to the rows of dy that no place names, by the first blocks of a gradient's grid: each looks
// for a window of rows through all places, while the other blocks work. (16384 rows of 8
// places: 32 blocks of 4096 rows, which read 16 MB from L2; no time that can be measured beside
// the 335 us of rows of 4096, where zeros for all rows first take 150 us. A call of a few rows
// takes 0.3 to 0.5 us longer. Blocks for cut rows, which live from L1, keep 1 KB of it for this.)
constexpr int ZERO_MIN_WINDOW = 1024, ZERO_MAX_WINDOW = 32768, ZERO_CUT_WINDOW = 8192, ZERO_MAX_BLOCKS = 2048;

template <bool ALIGNED>
__device__ __forceinline__ void zero_unnamed_rows(const RowsParams& p) {
  __shared__ uint32_t s_named[(ALIGNED ? ZERO_MAX_WINDOW : ZERO_CUT_WINDOW) / 32];
  constexpr int AT_ONCE = 8;  // words of places of a thread whose loads are in flight together
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, words = p.zero_window / 32;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.zero_window;
  for (int w = threadIdx.x; w < words; w += ROWS_THREADS) s_named[w] = 0;
  __syncthreads();
  const auto name = [&](int place) {
    const int64_t at = place - first;
    if (at >= 0 && at < p.zero_window) atomicOr(&s_named[at >> 5], 1u << (at & 31));
  };
  // whole 16-byte words of places, and the few before and behind them
  const int64_t head = min(p.entries, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(p.places) & 15)) & 15) >> 2));
  const int4* of4 = reinterpret_cast<const int4*>(p.places + head);
  const int64_t n4 = (p.entries - head) >> 2;
  for (int64_t i0 = threadIdx.x; i0 < n4; i0 += AT_ONCE * ROWS_THREADS) {
    int4 v[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int64_t i = i0 + k * ROWS_THREADS;
      v[k] = i < n4 ? of4[i] : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      name(v[k].x);
      name(v[k].y);
      name(v[k].z);
      name(v[k].w);
    }
  }
  if (threadIdx.x < head) name(p.places[threadIdx.x]);
  if (head + 4 * n4 + threadIdx.x < p.entries) name(p.places[head + 4 * n4 + threadIdx.x]);
  __syncthreads();
  for (int w = warp; w < words; w += ROWS_THREADS / 32) {  // a row to a warp
    for (uint32_t rest = ~s_named[w]; rest != 0; rest &= rest - 1) {
      const int64_t row = first + 32 * w + __ffs(rest) - 1;
      if (row >= p.x_rows) break;
      uint16_t* out = row_of(p.out, row, p.ldo);
      const uint4 zeros = make_uint4(0, 0, 0, 0);
      if constexpr (ALIGNED) {
        for (int c = 8 * lane; c < p.cols; c += 8 * 32) *reinterpret_cast<uint4*>(out + c) = zeros;
      } else {
        const CutRow cut(out, p.cols);
        for (int c = cut.body + 8 * lane; c < cut.tail; c += 8 * 32) *reinterpret_cast<uint4*>(out + c) = zeros;
        if (lane < cut.ends) out[cut.end(lane)] = 0;
      }
    }
  }
}

// Gradients of the sum by y and by the weights, a block to a row: a piece of
// dout is multiplied by each weight for dy, and by each row of y for dw.
template <bool BF16>
__global__ void __launch_bounds__(ROWS_THREADS) combine_rows_grad_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float s_sum[ROWS_THREADS / 32][ROWS_AT_ONCE];
  grid_dependency_wait();
  if (static_cast<int>(blockIdx.x) < p.zero_blocks) {
    zero_unnamed_rows<true>(p);
    return;
  }
  const int64_t row = static_cast<int64_t>(blockIdx.x) - p.zero_blocks;
  const uint16_t* dout = row_of(p.dout, row, p.ldd);
  const int32_t* places = p.places + row * p.top;
  const float* weights = p.weights ? p.weights + row * p.top : nullptr;
  for (int j0 = 0; j0 < p.top; j0 += ROWS_AT_ONCE) {
    int64_t at[ROWS_AT_ONCE];
    float w[ROWS_AT_ONCE], dot[ROWS_AT_ONCE];
#pragma unroll
    for (int j = 0; j < ROWS_AT_ONCE; ++j) {
      at[j] = j0 + j < p.top ? places[j0 + j] : -1;
      if (at[j] >= p.x_rows) at[j] = -1;
      w[j] = at[j] >= 0 && weights ? weights[j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    // one piece of dy and its part of dw
    const auto piece = [&](int j, uint16_t* dy, const float (&d)[8], const uint4& y) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = d[k] * w[j];
      *reinterpret_cast<uint4*>(dy) = pack_piece<BF16>(f);
      if (p.dweights) {
        unpack_piece<BF16>(y, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot[j] += d[k] * f[k];
      }
    };
    for (int c = 8 * threadIdx.x; c < p.cols; c += 8 * ROWS_THREADS) {
      float d[8];
      unpack_piece<BF16>(*reinterpret_cast<const uint4*>(dout + c), d);
      uint4 v[ROWS_AT_ONCE];
      if (p.dweights) {
#pragma unroll
        for (int j = 0; j < ROWS_AT_ONCE; ++j)
          if (at[j] >= 0) v[j] = *reinterpret_cast<const uint4*>(row_of(p.x, at[j], p.ldx) + c);
      }
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j)
        if (at[j] >= 0) piece(j, row_of(p.out, at[j], p.ldo) + c, d, v[j]);
    }
    if (p.dweights) {
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < ROWS_AT_ONCE && j0 + static_cast<int>(threadIdx.x) < p.top) {
        float sum = 0.0f;
        for (int k = 0; k < ROWS_THREADS / 32; ++k) sum += s_sum[k][threadIdx.x];
        p.dweights[row * p.top + j0 + threadIdx.x] = sum;
      }
      __syncthreads();
    }
  }
  grid_launch_dependents();
}

// The same for rows off 16-byte boundaries: a warp to an entry (several, each with a part of the
// columns, where there are fewer entries than warps), since each row of dy is cut elsewhere and
// takes dout in pieces of its own (from L1 for all but the first). Bound by latency: 16384
// rows of 4001 from 8 places take 420 us with two pieces at once and 8 blocks an SM, 443 us with
// four and 4, 500 us with one and 10; a block that goes through its entries in turn 530 us.
template <bool BF16>
__global__ void __launch_bounds__(ROWS_THREADS, 8) combine_rows_grad_cut_kernel(const __grid_constant__ RowsParams p) {
  constexpr int WARPS = ROWS_THREADS / 32, AT_ONCE = 2;  // pieces of a lane whose loads are in flight together
  __shared__ float s_sum[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = p.top == 1 ? WARPS : p.top == 2 ? WARPS / 2 : 1, entries = WARPS / parts;
  const int part = warp / entries;
  grid_dependency_wait();
  if (static_cast<int>(blockIdx.x) < p.zero_blocks) {
    zero_unnamed_rows<false>(p);
    return;
  }
  const int64_t row = static_cast<int64_t>(blockIdx.x) - p.zero_blocks;
  const uint16_t* dout = row_of(p.dout, row, p.ldd);
  const int32_t* places = p.places + row * p.top;
  const float* weights = p.weights ? p.weights + row * p.top : nullptr;
  for (int j = warp % entries; j < p.top; j += entries) {
    const int64_t at = places[j];
    float dot = 0.0f;
    if (at >= 0 && at < p.x_rows) {
      const float w = weights ? weights[j] : 1.0f;
      uint16_t* dy = row_of(p.out, at, p.ldo);
      // (without dw y is not read, and may not be there)
      const uint16_t* y = p.dweights ? row_of(p.x, at, p.ldx) : dout;
      const CutRow cut(dy, p.cols);
      const int end = part == 0 && lane < cut.ends ? cut.end(lane) : -1;
      uint16_t end_d = 0, end_y = 0;
      if (end >= 0) {
        end_d = dout[end];
        end_y = y[end];
      }
      for (int c0 = cut.body + 8 * (32 * part + lane); c0 < cut.tail; c0 += 8 * 32 * AT_ONCE * parts) {
        ShiftedPiece a[AT_ONCE], b[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
          const int c = c0 + 8 * 32 * parts * k;
          if (c >= cut.tail) continue;
          b[k] = load_words(y + c);
          a[k] = load_words(dout + c);
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
          const int c = c0 + 8 * 32 * parts * k;
          if (c >= cut.tail) continue;
          float d[8], f[8];
          unpack_piece<BF16>(shifted(a[k]), d);
          unpack_piece<BF16>(shifted(b[k]), f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot += d[i] * f[i];
            f[i] = d[i] * w;
          }
          *reinterpret_cast<uint4*>(dy + c) = pack_piece<BF16>(f);
        }
      }
      if (end >= 0) {
        const float d = to_float<BF16>(end_d);
        dot += d * to_float<BF16>(end_y);
        dy[end] = from_float<BF16>(d * w);
      }
    }
    if (p.dweights) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (parts == 1) {
        if (lane == 0) p.dweights[row * p.top + j] = dot;
      } else if (lane == 0) {
        s_sum[warp] = dot;
      }
    }
  }
  if (p.dweights && parts > 1) {  // (one entry a warp)
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < entries) {
      float sum = 0.0f;
      for (int k = 0; k < parts; ++k) sum += s_sum[k * entries + threadIdx.x];
      p.dweights[row * p.top + threadIdx.x] = sum;
    }
  }
  grid_launch_dependents();
}

}  // namespace sptg
