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
// All but the sort are bound by memory: each row is read once and written once,
// and `place` is a permutation, so that each row has one writer and nothing needs
// an atomic. Rows go through registers in pieces of 8 elements (16 bytes), or
// element by element where width, pitch or alignment forbid it.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace sptg {

constexpr int DISPATCH_MAX_EXPERTS = 1024;
constexpr int SORT_WARPS = 32;
constexpr int SORT_CLUSTER = 8;  // CTAs that share a long sort

struct SortParams {
  const int32_t* experts;  // entries
  int32_t* places;
  int32_t* offsets;        // E + 1
  int64_t entries;
  int64_t per_warp;        // entries of a warp, a multiple of 32
  int E;
};

// Counts by warp and expert, then one array for the totals of the CTA.
__host__ __device__ constexpr int sort_smem(int warps, int E) {
  return (warps + 1) * (E + 1) * 4;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Stable sort of the entries by expert, by counting: one cluster of CTAs. Every
// warp has a run of neighbouring entries of its own, counts them by expert, learns
// from the other warps and CTAs how many entries go before its own of each expert,
// and goes through its run once more to hand out the places. No atomics: a warp
// takes 32 entries at a time, and the lanes of equal experts find each other.
template <int SORT_WARPS>
__global__ void __launch_bounds__(32 * SORT_WARPS) dispatch_sort_kernel(const SortParams p) {
  extern __shared__ uint32_t counts[];  // [SORT_WARPS][bins], then the CTA's totals
  __shared__ uint32_t s_warp[SORT_WARPS];
  const int bins = p.E + 1;  // (the last: entries of no expert)
  uint32_t* totals = counts + SORT_WARPS * bins;
  constexpr int SORT_THREADS = 32 * SORT_WARPS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
  for (int i = threadIdx.x; i < SORT_WARPS * bins; i += SORT_THREADS) counts[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  uint32_t* mine = counts + warp * bins;
  const int64_t begin = (static_cast<int64_t>(rank) * SORT_WARPS + warp) * p.per_warp;
  const int64_t end = min(p.entries, begin + p.per_warp);
  const auto bin_of = [&](int64_t i) {
    const int e = p.experts[i];
    return e < 0 || e >= p.E ? p.E : e;
  };
  for (int64_t i = begin + lane; i - lane < end; i += 32) {
    const int b = i < end ? bin_of(i) : bins;
    const uint32_t same = __match_any_sync(0xffffffffu, b);
    if (i < end && lane == __ffs(same) - 1) mine[b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // entries of each expert in the warps before, and in the CTA
  for (int b = threadIdx.x; b < bins; b += SORT_THREADS) {
    uint32_t sum = 0;
    for (int w = 0; w < SORT_WARPS; ++w) {
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
  if (e < p.E) {
    const uint32_t at = smem_addr(totals + e);
    for (int c = 0; c < ctas; ++c) {
      const uint32_t n = ld_cluster_u32(map_to_cta(at, c));
      if (c < rank) before += n;
      all += n;
    }
  }
  uint32_t none_before = 0;  // (of entries of no expert)
  for (int c = 0; c < rank; ++c) none_before += ld_cluster_u32(map_to_cta(smem_addr(totals + p.E), c));
  // where each expert starts
  uint32_t sum = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  uint32_t base = 0, live = 0;
  for (int w = 0; w < SORT_WARPS; ++w) {
    const uint32_t n = s_warp[w];
    if (w < warp) base += n;
    live += n;
  }
  const uint32_t start = base + sum - all;
  if (rank == 0) {
    if (e < p.E) p.offsets[e] = static_cast<int32_t>(start);
    if (e == 0) p.offsets[p.E] = static_cast<int32_t>(live);
  }
  if (e < p.E)
    for (int w = 0; w < SORT_WARPS; ++w) counts[w * bins + e] += start + before;
  if (e < SORT_WARPS) counts[e * bins + p.E] += live + none_before;
  cluster_sync();  // (the totals have been read, and this CTA's counts are places now)
  grid_launch_dependents();
  for (int64_t i = begin + lane; i - lane < end; i += 32) {
    const int b = i < end ? bin_of(i) : bins;
    const uint32_t same = __match_any_sync(0xffffffffu, b);
    uint32_t place = 0;
    if (i < end) place = mine[b] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (i < end) {
      p.places[i] = static_cast<int32_t>(place);
      if (lane == __ffs(same) - 1) mine[b] += __popc(same);
    }
    __syncwarp();
  }
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
};

constexpr int ROWS_THREADS = 128;
constexpr int ROWS_AT_ONCE = 8;  // entries of a row whose loads are in flight together

template <int VEC>
struct RowPiece {
  uint4 v;
};
template <>
struct RowPiece<1> {
  uint16_t v;
};

template <int VEC>
__device__ __forceinline__ RowPiece<VEC> load_piece(const void* base, int64_t row, int64_t ld, int i) {
  RowPiece<VEC> r;
  const uint16_t* p = static_cast<const uint16_t*>(base) + row * ld;
  if constexpr (VEC == 8)
    r.v = reinterpret_cast<const uint4*>(p)[i];
  else
    r.v = p[i];
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_piece(void* base, int64_t row, int64_t ld, int i,
                                            const RowPiece<VEC>& r) {
  uint16_t* p = static_cast<uint16_t*>(base) + row * ld;
  if constexpr (VEC == 8)
    reinterpret_cast<uint4*>(p)[i] = r.v;
  else
    p[i] = r.v;
}

template <bool BF16, int VEC>
__device__ __forceinline__ void unpack_piece(const RowPiece<VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 8) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
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
  } else if constexpr (BF16) {
    f[0] = __uint_as_float(static_cast<uint32_t>(r.v) << 16);
  } else {
    f[0] = __half2float(__ushort_as_half(r.v));
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ RowPiece<VEC> pack_piece(const float (&f)[VEC]) {
  constexpr int OUT = BF16 ? OUT_BF16 : OUT_F16;
  RowPiece<VEC> r;
  if constexpr (VEC == 8)
    r.v = make_uint4(pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]), pack2<OUT>(f[4], f[5]),
                     pack2<OUT>(f[6], f[7]));
  else
    r.v = static_cast<uint16_t>(pack2<OUT>(f[0], 0.0f));
  return r;
}

// Rows of x to their places: a block to a row and a part of its columns
// (blockIdx.y). A place outside of the sorted rows is passed over.
template <int VEC>
__global__ void __launch_bounds__(ROWS_THREADS) dispatch_copy_kernel(const RowsParams p) {
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const int pieces = p.cols / VEC;
  const int32_t* places = p.places + row * p.top;
  for (int i = blockIdx.y * ROWS_THREADS + threadIdx.x; i < pieces; i += gridDim.y * ROWS_THREADS) {
    const RowPiece<VEC> v = load_piece<VEC>(p.x, row, p.ldx, i);
    for (int j = 0; j < p.top; ++j) {
      const int64_t to = places[j];
      if (to >= 0 && to < p.out_rows) store_piece<VEC>(p.out, to, p.ldo, i, v);
    }
  }
  grid_launch_dependents();
}

// Sums of the rows that a row's places name, in 32 bits and in the order of the
// places, rounded once. A place outside of y counts as a row of zeros.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(ROWS_THREADS) combine_rows_kernel(const RowsParams p) {
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const int pieces = p.cols / VEC;
  const int32_t* places = p.places + row * p.top;
  const float* weights = p.weights ? p.weights + row * p.top : nullptr;
  for (int i = blockIdx.y * ROWS_THREADS + threadIdx.x; i < pieces; i += gridDim.y * ROWS_THREADS) {
    float sum[VEC];
    if (p.base) {
      unpack_piece<BF16, VEC>(load_piece<VEC>(p.base, row, p.ldb, i), sum);
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) sum[c] = 0.0f;
    }
    for (int j0 = 0; j0 < p.top; j0 += ROWS_AT_ONCE) {
      RowPiece<VEC> v[ROWS_AT_ONCE];
      float w[ROWS_AT_ONCE];
      bool in[ROWS_AT_ONCE];
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j) {
        const int64_t from = j0 + j < p.top ? places[j0 + j] : -1;
        in[j] = from >= 0 && from < p.x_rows;
        w[j] = in[j] && weights ? weights[j0 + j] : 1.0f;
        if (in[j]) v[j] = load_piece<VEC>(p.x, from, p.ldx, i);
      }
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j) {
        if (!in[j]) continue;
        float f[VEC];
        unpack_piece<BF16, VEC>(v[j], f);
#pragma unroll
        for (int c = 0; c < VEC; ++c) sum[c] += w[j] * f[c];
      }
    }
    store_piece<VEC>(p.out, row, p.ldo, i, pack_piece<BF16, VEC>(sum));
  }
  grid_launch_dependents();
}

// Gradients of the sum by y and by the weights, a block to a row: a piece of
// dout is multiplied by each weight for dy, and by each row of y for dw.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(ROWS_THREADS) combine_rows_grad_kernel(const RowsParams p) {
  __shared__ float s_sum[ROWS_THREADS / 32][ROWS_AT_ONCE];
  const int64_t row = blockIdx.x;
  grid_dependency_wait();
  const int pieces = p.cols / VEC;
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
    for (int i = threadIdx.x; i < pieces; i += ROWS_THREADS) {
      float d[VEC];
      unpack_piece<BF16, VEC>(load_piece<VEC>(p.dout, row, p.ldd, i), d);
      RowPiece<VEC> v[ROWS_AT_ONCE];
      if (p.dweights) {
#pragma unroll
        for (int j = 0; j < ROWS_AT_ONCE; ++j)
          if (at[j] >= 0) v[j] = load_piece<VEC>(p.x, at[j], p.ldx, i);
      }
#pragma unroll
      for (int j = 0; j < ROWS_AT_ONCE; ++j) {
        if (at[j] < 0) continue;
        float f[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) f[c] = d[c] * w[j];
        store_piece<VEC>(p.out, at[j], p.ldo, i, pack_piece<BF16, VEC>(f));
        if (p.dweights) {
          unpack_piece<BF16, VEC>(v[j], f);
#pragma unroll
          for (int c = 0; c < VEC; ++c) dot[j] += d[c] * f[c];
        }
      }
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

}  // namespace sptg
