// grouped_gemm.cuh -- products grouped by expert with ragged sizes, and their
// gradients, on CTA pairs with the 2-SM tensor-core instruction.
//
// Rows offsets[e] ... offsets[e + 1] - 1 of X (and of Y, dY, dX) belong to
// expert e, whose weights are W[e] (N x K):
//
//   GROUPED_Y    Y[t, n]     = sum_k X[t, k]  W[e, n, k]
//   GROUPED_DX   dX[t, k]    = sum_n dY[t, n] W[e, n, k]
//   GROUPED_DW   dW[e, n, k] = sum_t dY[t, n] X[t, k]     (t over e's rows)
//
// The offsets are read on the device, so a caller never waits for the GPU to
// learn the sizes: the grid is fixed (persistent CTA pairs) and every CTA works
// out the same list of tiles from the offsets.
//
// Orientation: the ragged side is the MMA's N side. The MMA's M side (256 over
// a pair: 128 of each CTA) covers "features" -- rows n of W (Y), columns k of
// W (dX), columns n of dY (dW) -- which are wide and regular; its N side
// covers up to TT rows of an expert (Y, dX), whose width the instruction takes
// in steps of 16. An expert with few rows so pays for few rows, and its weights
// stream through the fixed 128-row side; on the other orientation it would pay
// for 128 or 256 rows. For dW the N side covers 256 columns k and the ragged
// side is the sum.
//
// Operands as they lie in memory, no transposed copies: the tensor core reads
// K-major tiles (rows contiguous along the sum: W and X for Y, dY for dX) and
// MN-major tiles (rows contiguous along the features: W for dX, both operands
// of dW), both 128-byte swizzled as the tensor-copy engine writes them.
//
// Bounds: rows of X past an expert's end that a tile's copy brings along only
// reach accumulator columns that are never stored. W is a 3-D tensor, so that
// a tile past its N or K reads zeros, not the next expert's weights. For dW
// the sum itself is ragged: the ring's MMAs stop at a multiple of 16 of an
// expert's rows, and a warp of its own gathers the up to 15 rows left, zeros
// below them, into a small operand tile for one last step (0 times another
// expert's infinity would be NaN, so neither operand may hold its rows). That
// tile is ready long before the step; clearing the rows in the ring's last
// stage instead made every tile wait for it (16 experts of 1000 rows, 4096 x
// 4096: 368 us against 320 with 1024 rows).
//
// Roles of a CTA: warp 0 producer, warp 1 MMA issuer (leader CTA only), warps
// 2-9 epilogue, warp 10 the rows left over (dW only). Two accumulators of up to 256 columns,
// so a tile's epilogue overlaps the next tile's K-loop.
//
// Measured (bf16, 16 experts of 4096 x 4096, 16384 rows): Y and dX 305 us (1800
// TFLOP/s of the 1926 that a dense product was measured at), dW 319 us: tensor-bound. 8192
// binary16 rows through 64 experts of 2048 x 4096: Y 185 us, 6.3 TB/s of weights,
// rows and output: memory-bound, as are 32 rows through those of 16 experts of 4096 x
// 2048 that they reach (Y 31 us). 1531 binary16 rows in 24 ragged experts of 1112 x
// 2056, f32 out: Y 33 us, dW 55 us, most of it the writing of 220 MB; dX 27 us.
//
// The epilogue reads its whole share of an accumulator into registers and hands
// it back before it converts and stores. That of Y and dX writes the transpose
// of the accumulator: a lane holds one feature, its columns are rows of the
// output. Each warp turns blocks of 32 x 32 in shared memory and stores rows of
// 32 features (a tensor copy could not stop at an expert's last row). dW's rows
// are features, so its blocks go out by tensor copy, which clips them at N and K.
#pragma once

#include "common.cuh"
#include "variants.h"

namespace sptg {

enum GroupedMode : int { GROUPED_Y = 0, GROUPED_DX = 1, GROUPED_DW = 2 };

constexpr int GROUPED_MAX_EXPERTS = 1024;
constexpr int GROUPED_EPI_WARPS = 8;  // two for each quarter of tensor memory's lanes
constexpr int GROUPED_THREADS = 32 * (2 + GROUPED_EPI_WARPS + 1);

struct GroupedParams {
  int experts;
  int T;   // rows of X
  int F;   // features (M side): N (Y, dW) or K (dX)
  int C;   // Y, dX: length of the sum (K, N); dW: columns of the output (K)
  const int32_t* offsets;  // experts + 1
  const uint16_t* a;       // dW: dY and X, for the rows left over, and their
  const uint16_t* b;       // row pitches
  int64_t lda, ldb;
  void* out;
  int64_t ldo;             // elements between output rows (Y, dX)
  int keep_weights;        // 1: W is read by several tiles; 0: once (evict first)
  unsigned int* error_word;
  uint64_t timeout_ns;
};

// TT: widest N side of a tile (256, or 64 for experts of few rows: the ring
// then holds eight or nine stages of weights).
template <int MODE, int TT, int OBYTES>
struct GroupedLayout {
  static constexpr int A_STAGE = 128 * 128;         // 128 features x 64 of the sum
  static constexpr int B_STAGE = TT / 2 * 128;      // this CTA's half of the N side
  static constexpr int STAGE = A_STAGE + B_STAGE;
  // as many as fit beside the epilogue's blocks
  static constexpr int STAGES = TT == 64             ? (OBYTES == 4 ? 8 : 9)
                                : MODE == GROUPED_DW ? 5
                                                     : (OBYTES == 4 ? 5 : 6);
  static constexpr int EPI_PITCH = 32 * OBYTES + 16;
  // an epilogue warp's block of 32 x 32; dW: of 32 rows of 128 bytes
  static constexpr int EPI_BUF = MODE == GROUPED_DW ? 4096 : 32 * EPI_PITCH;
  static constexpr int OFF_EPI = STAGES * STAGE;
  // dW: two operand tiles of the rows left over, 16 lines of 128 features and
  // of 128 columns each
  static constexpr int TAIL = 16 * 128 * 4;
  static constexpr int OFF_TAIL = OFF_EPI + GROUPED_EPI_WARPS * EPI_BUF;
  static constexpr int OFF_BAR = OFF_TAIL + (MODE == GROUPED_DW ? 2 * TAIL : 0);
  static constexpr int NUM_BARS = 2 * STAGES + 9;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_GROUPS = OFF_MISC + 16;
  // first row and first tile of each expert, of the rows before the first
  // expert and after the last (written as zeros), and of the end
  static constexpr int GROUP_SLOTS = GROUPED_MAX_EXPERTS + 3;
  static constexpr int BYTES_USED = OFF_GROUPS + 3 * GROUP_SLOTS * 4;
  static constexpr int SMEM_BYTES = BYTES_USED + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget exceeded");
};

// Matrix descriptor of an MN-major operand tile: lines of 64 elements (128
// bytes, swizzled) along the M or N side, one line for each step of the sum,
// 8-line groups 1024 bytes apart, the next 64 elements `atom` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_major_sw128(uint32_t saddr, uint32_t atom) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(atom >> 4) << 16;   // leading byte offset: next 64 elements
  d |= static_cast<uint64_t>(1024u >> 4) << 32;  // stride byte offset: next 8 of the sum
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// The MMA's N side for `n` rows or columns: steps of 32, and of 16 past 96
// (the widths of 112 and more that the square kernel's pair tiles use).
__host__ __device__ constexpr int grouped_mma_n(int n) {
  return n <= 96 ? (n + 31) & ~31 : (n + 15) & ~15;
}

// Pieces of 64 of a sum that one accumulator takes (a power of two). The tensor
// core cuts off what an addition shifts out, so an error grows with the length of
// a sum and has one sign: relative 4.7e-6 after 4000 rows of binary16. A 16-bit
// output does not show it (2e-4); for a 32-bit output the accumulator is read after
// 512 of the sum (256 in sums up to 1024) and the parts are added up, rounded to
// nearest, in the epilogue's registers: 6e-7 at any length, where 32-bit additions
// one by one leave 1.1e-6. 16384 rows of 16 experts, 4096 x 4096, f32 out: Y 340 us
// against 330 with one accumulator, dW 444 against 380 (with 256 throughout 443 and
// 513: while the epilogue stores a tile the next one has two accumulators to go on).
__device__ __forceinline__ int grouped_span(int out, int chunks) {
  return out != OUT_F32 ? 1 << 26 : chunks > 16 ? 8 : 4;
}

// One tile of work.
struct GroupedTile {
  int e;       // expert
  int f0;      // first feature
  int t0;      // Y, dX: first row of the tile; dW: the expert's first row
  int rows;    // Y, dX: rows of the tile; dW: rows of the expert
  int c0;      // dW: first column
  int n;       // width of the MMA's N side
  int chunks;  // 64-long pieces of the sum in the ring
  int steps;   // steps of 16 of the last of them
  int tail;    // dW: rows left over, 0 ... 15
  __device__ __forceinline__ bool zeros() const { return chunks == 0 && tail == 0; }
};

template <int MODE, int TT>
struct GroupedSchedule {
  const int* first;  // in shared memory: first row
  const int* count;  // rows
  const int* cum;    // tiles before the group
  int groups, nf, F, C;
  int g = 0;

  __device__ __forceinline__ int total() const { return cum[groups]; }

  // `tile` never decreases from call to call
  __device__ __forceinline__ GroupedTile at(int tile) {
    while (tile >= cum[g + 1]) ++g;
    GroupedTile w;
    const int i = tile - cum[g];
    const int first_g = first[g], count_g = count[g];
    w.e = g;
    if constexpr (MODE == GROUPED_DW) {
      const int nc = (C + 255) >> 8;
      int ft, ct;
      tile_coords(i, nf, nc, 8, ft, ct);
      w.f0 = ft * 256;
      w.c0 = ct * 256;
      w.t0 = first_g;
      w.rows = count_g;
      w.n = grouped_mma_n(min(256, C - w.c0));
      w.chunks = (count_g + 48) >> 6;  // of the whole steps of 16
      w.steps = count_g < 16 ? 0 : ((((count_g >> 4) - 1) & 3) + 1);
      w.tail = count_g & 15;
    } else {
      const int nt = (count_g + TT - 1) / TT;
      // the expert's rows in tiles of equal width (a multiple of 16)
      const int width = ((count_g + nt - 1) / nt + 15) & ~15;
      int tt, ft;
      tile_coords(i, nt, nf, 8, tt, ft);
      w.f0 = ft * 256;
      w.c0 = 0;
      w.t0 = first_g + tt * width;
      w.rows = max(0, min(width, first_g + count_g - w.t0));
      w.n = grouped_mma_n(w.rows);
      // groups past the experts are rows that belong to none
      w.chunks = (g < groups - 2 && w.rows > 0) ? (C + 63) >> 6 : 0;
      w.steps = 4;  // (past C both operands read zeros)
      w.tail = 0;
    }
    return w;
  }
};

template <int MODE, int TT, bool BF16, int OUT>
__global__ void __launch_bounds__(GROUPED_THREADS, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmA,   // the features' operand
                        const __grid_constant__ CUtensorMap tmB,   // the N side, boxes of 32 rows
                        // the N side in boxes of 128 rows; dW: the output
                        const __grid_constant__ CUtensorMap tmB4,
                        const GroupedParams p) {
  constexpr int OBYTES = OutTraits<OUT>::bytes;
  using L = GroupedLayout<MODE, TT, OBYTES>;
  constexpr int STAGES = L::STAGES;
  constexpr bool A_MN = MODE != GROUPED_Y, B_MN = MODE == GROUPED_DW;
  static_assert(MODE != GROUPED_DW || TT == 256, "dW tiles are 256 columns wide");
  constexpr uint32_t IDESC0 = idesc_f16_f32acc(BF16, 256, 0) | (A_MN ? 1u << 15 : 0u) |
                              (B_MN ? 1u << 16 : 0u);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  auto stage_a = [&](int s) { return sbase + s * L::STAGE; };
  auto stage_b = [&](int s) { return sbase + s * L::STAGE + L::A_STAGE; };
  const uint32_t bar0 = sbase + L::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  auto rest_full = [&](int b) { return bar0 + 8u * (2 * STAGES + 4 + b); };   // dW: rows left over
  auto rest_empty = [&](int b) { return bar0 + 8u * (2 * STAGES + 6 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 8);
  auto rest_tile = [&](int b) { return sbase + L::OFF_TAIL + b * L::TAIL; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  int* g_first = reinterpret_cast<int*>(smem + L::OFF_GROUPS);
  int* g_count = g_first + L::GROUP_SLOTS;
  int* g_cum = g_count + L::GROUP_SLOTS;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int worker = static_cast<int>(blockIdx.x >> 1);
  const int workers = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 2 * GROUPED_EPI_WARPS);  // of both CTAs
      mbar_init(rest_full(b), 2);                       // both CTAs' halves
      mbar_init(rest_empty(b), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensor_map(&tmA);
    prefetch_tensor_map(&tmB);
    prefetch_tensor_map(&tmB4);
  }
  if (warp == 1) {
    tmem_alloc_g<true>(smem_addr(tmem_slot), 512);
    tmem_relinquish_g<true>();
  }
  grid_dependency_wait();
  // The list of groups: experts 0 ... experts - 1, then the rows before the
  // first and after the last. Offsets outside [0, T] are clamped to it and
  // smaller ones raised to the largest before them, so that no tile leaves the
  // rows of X and each row belongs to one group.
  const int groups = MODE == GROUPED_DW ? p.experts : p.experts + 2;
  const int nf = (p.F + 255) >> 8;
  if (warp == 2) {
    const int lo = min(max(p.offsets[0], 0), p.T);
    int base = 0, before = 0;  // tiles, and the largest offset, of the groups so far
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      // where a group starts: the largest offset up to its own
      int start = g <= p.experts ? min(max(p.offsets[g], 0), p.T) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, start, o);
        if (lane >= o) start = max(start, up);
      }
      start = max(start, before);
      before = __shfl_sync(0xffffffffu, start, 31);
      int a = 0, n = 0, tiles = 0;
      if (g < groups) {
        if (g < p.experts) {
          a = start;
          n = max(min(p.offsets[g + 1], p.T), start) - start;
        } else if (g == p.experts) {
          n = lo;
        } else {
          a = start;  // (the last expert's end)
          n = p.T - start;
        }
        tiles = MODE == GROUPED_DW ? nf * ((p.C + 255) >> 8) : (n + TT - 1) / TT * nf;
      }
      int sum = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (g < groups) {
        g_first[g] = a;
        g_count[g] = n;
        g_cum[g] = base + sum - tiles;
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) g_cum[groups] = base;
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  GroupedSchedule<MODE, TT> sched{g_first, g_count, g_cum, groups, nf, p.F, p.C};
  const int total = sched.total();
  const WaitCtl ctl{p.timeout_ns, p.error_word, abort_flag};

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one_sync();
    const uint64_t pol_a = p.keep_weights ? policy_evict_last() : policy_evict_first();
    const uint64_t pol_b = policy_evict_last();
    int s = 0;
    uint32_t round = 0;
    int issued = 0;
    bool ok = true;
    for (int tile = worker; ok && tile < total; tile += workers) {
      const GroupedTile w = sched.at(tile);
      const int half = w.n >> 1;
      const int n_first = static_cast<int>(rank) * half;  // this CTA's part of the N side
      // boxes of the N side and the bytes of one stage (both CTAs)
      const int boxes = MODE == GROUPED_DW ? (half + 63) >> 6 : (half + 31) >> 5;
      const uint32_t own_tx =
          L::A_STAGE + static_cast<uint32_t>(boxes) * (MODE == GROUPED_DW ? 8192u : 4096u);
      const int f = w.f0 + 128 * static_cast<int>(rank);
      for (int c = 0; c < w.chunks; ++c) {
        if (round > 0 && !__all_sync(0xffffffffu, wait_bounded_lazy(empty_bar(s), (round & 1u) ^ 1u,
                                                                ctl, WAIT_PRODUCER_EMPTY))) {
          ok = false;
          break;
        }
        ++issued;
        if (leader) {
          const uint32_t a = stage_a(s), b = stage_b(s);
          if constexpr (MODE == GROUPED_DW) {
            const int t = w.t0 + 64 * c;
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * own_tx);
            const uint32_t full = map_to_cta(full_bar(s), 0u);
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(a + j * 8192, &tmA, full, f + 64 * j, t, pol_b);
            for (int j = 0; j < boxes; ++j)
              tma_load_2d_pair(b + j * 8192, &tmB, full, w.c0 + n_first + 64 * j, t, pol_b);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * own_tx);
            const uint32_t full = map_to_cta(full_bar(s), 0u);
            if constexpr (MODE == GROUPED_Y) {
              tma_load_3d_pair(a, &tmA, full, 64 * c, f, w.e, pol_a);
            } else {
              for (int j = 0; j < 2; ++j)
                tma_load_3d_pair(a + j * 8192, &tmA, full, f + 64 * j, 64 * c, w.e, pol_a);
            }
            if (boxes == 4) {
              tma_load_2d_pair(b, &tmB4, full, 64 * c, w.t0 + n_first, pol_b);
            } else {
              for (int j = 0; j < boxes; ++j)
                tma_load_2d_pair(b + j * 4096, &tmB, full, 64 * c, w.t0 + n_first + 32 * j, pol_b);
            }
          }
        }
        if (++s == STAGES) {
          s = 0;
          ++round;
        }
      }
    }
    grid_launch_dependents();
    if (!ok) {
      // let every copy already issued land before the CTA can exit
      if (leader && rank == 0) {
        for (int i = max(0, issued - STAGES); i < issued; ++i) {
          const uint32_t bar = full_bar(i % STAGES);
          const uint32_t par = static_cast<uint32_t>(i / STAGES) & 1u;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(bar, par) && global_timer_ns() - t0 < ctl.timeout_ns) {
          }
        }
      }
      __syncwarp();
      if (rank != 0) {
        // copies that complete on the leader's barriers, which this CTA
        // cannot wait on: give them a fixed 100 us to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (rank == 0) {
      const bool leader = elect_one_sync();
      int s = 0;
      uint32_t phase = 0, unit = 0, rest = 0;
      bool ok = true;
      for (int tile = worker; ok && tile < total; tile += workers) {
        const GroupedTile w = sched.at(tile);
        if (w.zeros()) continue;
        uint32_t b, d;
        auto next_accumulator = [&]() {
          b = unit & 1u;
          d = tmem_base + b * 256;
          ok = __all_sync(0xffffffffu, wait_bounded_lazy(tempty_bar(b), ((unit >> 1) & 1u) ^ 1u, ctl,
                                                         WAIT_MMA_TMEM_EMPTY));
          ++unit;
          tc_fence_after();
          return ok;
        };
        if (!next_accumulator()) break;
        const int span = grouped_span(OUT, w.chunks);
        const uint32_t idesc = IDESC0 | (static_cast<uint32_t>(w.n >> 3) << 17);
        for (int c = 0; c < w.chunks; ++c) {
          if (c > 0 && (c & (span - 1)) == 0) {
            if (leader) mma_commit_g<true>(tfull_bar(b));
            __syncwarp();
            if (!next_accumulator()) break;
          }
          if (!__all_sync(0xffffffffu, wait_bounded_lazy(full_bar(s), phase, ctl, WAIT_MMA_FULL))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            const uint64_t ad = A_MN ? sdesc_mn_major_sw128(stage_a(s), 8192)
                                     : sdesc_k_major_sw128(stage_a(s));
            const uint64_t bd = B_MN ? sdesc_mn_major_sw128(stage_b(s), 8192)
                                     : sdesc_k_major_sw128(stage_b(s));
            // one step of 16 along the sum: 32 bytes of a K-major row, 16
            // lines of an MN-major tile (in units of 16 bytes)
            constexpr uint64_t ADV_A = A_MN ? 128 : 2, ADV_B = B_MN ? 128 : 2;
            const int steps = c == w.chunks - 1 ? w.steps : 4;
            mma_f16_g<true>(d, ad, bd, idesc, (c & (span - 1)) != 0 ? 1u : 0u);
#pragma unroll
            for (int k = 1; k < 4; ++k)
              if (MODE != GROUPED_DW || steps > k)
                mma_f16_g<true>(d, ad + ADV_A * k, bd + ADV_B * k, idesc, 1u);
            mma_commit_g<true>(empty_bar(s));
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (MODE == GROUPED_DW && ok && w.tail != 0) {
          const uint32_t rb = rest & 1u;
          ok = __all_sync(0xffffffffu,
                          wait_bounded_lazy(rest_full(rb), (rest >> 1) & 1u, ctl, WAIT_MMA_FULL));
          ++rest;
          tc_fence_after();
          if (ok && leader) {
            mma_f16_g<true>(d, sdesc_mn_major_sw128(rest_tile(rb), 2048),
                            sdesc_mn_major_sw128(rest_tile(rb) + 4096, 2048), idesc,
                            w.chunks > 0 ? 1u : 0u);
            mma_commit_g<true>(rest_empty(rb));
          }
          __syncwarp();
        }
        if (ok && leader) mma_commit_g<true>(tfull_bar(b));
        __syncwarp();
      }
      if (leader) mma_commit_local_g<true>(drain_bar);
      __syncwarp();
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain_bar, 0) && global_timer_ns() - t0 < ctl.timeout_ns) {
      }
    }
  } else if (warp < 2 + GROUPED_EPI_WARPS) {
    // ------------------------------------------------------------ epilogue
    // lanes 32q ... 32q + 31 of tensor memory, every second block of columns
    const int q = warp & 3, part = (warp - 2) >> 2;
    uint8_t* buf = smem + L::OFF_EPI + (warp - 2) * L::EPI_BUF;
    constexpr int PITCH = L::EPI_PITCH;
    constexpr int VEC = 16 / OBYTES;            // outputs in 16 bytes
    constexpr int VPR = 32 / VEC;               // 16-byte pieces of a row of 32
    constexpr int RPI = 32 / VPR;               // rows a warp stores at a time
    const int vr = lane / VPR, vc = lane % VPR;
    // this warp's blocks of 32 columns: dW takes two neighbours in turn
    constexpr int NB = TT / 64;
    constexpr bool SUMS = OUT == OUT_F32;  // a tile's accumulators are added up here
    auto block_col = [&](int i) {
      return MODE == GROUPED_DW ? (i >> 1) * 128 + part * 64 + (i & 1) * 32 : 64 * i + 32 * part;
    };
    uint32_t unit = 0;
    for (int tile = worker; tile < total; tile += workers) {
      const GroupedTile w = sched.at(tile);
      const int f = w.f0 + 128 * static_cast<int>(rank) + 32 * q;  // this warp's first feature
      uint32_t r[NB][32];
      if (SUMS || w.zeros()) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int k = 0; k < 32; ++k) r[i][k] = 0;
      }
      bool ok = true;
      const int span = grouped_span(OUT, w.chunks);
      for (int c = 0; !w.zeros() && (c == 0 || c < w.chunks); c += span) {
        const uint32_t b = unit & 1u;
        ok = __all_sync(0xffffffffu, wait_bounded_lazy(tfull_bar(b), (unit >> 1) & 1u, ctl,
                                                       WAIT_EPI_TMEM_FULL));
        if (!ok) break;
        ++unit;
        tc_fence_after();
        const uint32_t t_acc = tmem_base + b * 256 + (static_cast<uint32_t>(32 * q) << 16);
        // (columns past the tile's width hold an earlier tile's sums, or
        // anything: they are not stored)
        if constexpr (SUMS) {
#pragma unroll
          for (int i = 0; i < 2 * NB; ++i) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_acc + block_col(i >> 1) + 16 * (i & 1), v);
            tmem_wait_ld_regs16(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              uint32_t& sum = r[i >> 1][16 * (i & 1) + k];
              sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(v[k]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NB; ++i) tmem_ld_32x32b_x32(t_acc + block_col(i), r[i]);
#pragma unroll
          for (int i = 0; i < NB; ++i) tmem_wait_ld_regs(r[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_cta(tempty_bar(b), 0u));
      }
      if (!ok) break;
      if (f >= p.F) continue;
      if constexpr (MODE == GROUPED_DW) {
        // blocks of 32 features x 128 bytes, in the tensor copy's swizzle
        constexpr int BLOCKS = 128 / OBYTES / 32;  // of 32 columns in 128 bytes
#pragma unroll
        for (int i = 0; i < NB; i += BLOCKS) {
          const int col = w.c0 + block_col(i);
          if (col >= p.C) break;
          if (lane == 0) bulk_wait_group_read<0>();  // the block before has been read
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 o;
            if constexpr (OBYTES == 4) {
              o = make_uint4(r[i][4 * j], r[i][4 * j + 1], r[i][4 * j + 2], r[i][4 * j + 3]);
            } else {
              const uint32_t* v = &r[i + j / 4][8 * (j % 4)];
              o = make_uint4(pack2<OUT>(__uint_as_float(v[0]), __uint_as_float(v[1])),
                             pack2<OUT>(__uint_as_float(v[2]), __uint_as_float(v[3])),
                             pack2<OUT>(__uint_as_float(v[4]), __uint_as_float(v[5])),
                             pack2<OUT>(__uint_as_float(v[6]), __uint_as_float(v[7])));
            }
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) = o;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmB4, smem_addr(buf), col, f, w.e);
            bulk_commit_group();
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int cb = block_col(i);
          if (cb >= w.rows) break;
          __syncwarp();  // the block before this one has been read
          // rows of the output are accumulator columns
#pragma unroll
          for (int k = 0; k < 32; ++k)
            store_out<OUT>(buf + k * PITCH, lane, __uint_as_float(r[i][k]));
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 32; k += RPI) {
            const uint4 v = *reinterpret_cast<const uint4*>(buf + (k + vr) * PITCH + 16 * vc);
            const int row = cb + k + vr, col = f + vc * VEC;
            const int64_t at = static_cast<int64_t>(w.t0 + row) * p.ldo + col;
            if (row < w.rows && col < p.F)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at * OBYTES) = v;
          }
        }
      }
    }
    if (MODE == GROUPED_DW && lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  } else if constexpr (MODE == GROUPED_DW) {
    // ------------------------------------------------------ rows left over
    // Gathers an expert's last rows (past the multiple of 16) for this CTA's
    // 128 features and its half of the columns: lines of 64 values in the
    // swizzle of the ring's tiles, zeros past the last row and the tensors.
    uint32_t rest = 0;
    for (int tile = worker; tile < total; tile += workers) {
      const GroupedTile w = sched.at(tile);
      if (w.tail == 0) continue;
      const uint32_t rb = rest & 1u;
      if (!__all_sync(0xffffffffu, wait_bounded_lazy(rest_empty(rb), ((rest >> 1) & 1u) ^ 1u, ctl,
                                                     WAIT_PRODUCER_EMPTY)))
        break;
      ++rest;
      const int64_t row0 = w.t0 + w.rows - w.tail;
      const int half = w.n >> 1;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const uint16_t* src = side == 0 ? p.a : p.b;
        const int64_t ld = side == 0 ? p.lda : p.ldb;
        const int col0 = side == 0 ? w.f0 + 128 * static_cast<int>(rank)
                                   : w.c0 + half * static_cast<int>(rank);
        const int limit = side == 0 ? p.F : min(p.C, col0 + half);
        uint4 v[8];
        // 16 lines of 16 pieces of 8 values: 8 pieces a lane
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int line = 2 * i + (lane >> 4), col = col0 + 8 * (lane & 15);
          v[i] = line < w.tail && col < limit
                     ? *reinterpret_cast<const uint4*>(src + (row0 + line) * ld + col)
                     : make_uint4(0, 0, 0, 0);
        }
        uint8_t* dst = smem + L::OFF_TAIL + rb * L::TAIL + side * 4096 + ((lane & 15) >> 3) * 2048;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int line = 2 * i + (lane >> 4);
          *reinterpret_cast<uint4*>(dst + line * 128 + (((lane & 7) ^ (line & 7)) << 4)) = v[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_cta(rest_full(rb), 0u));
    }
  }

  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the pair's MMAs may still read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_g<true>(tmem_base, 512);
  }
}

template <int MODE, int TT, bool BF16, int OUT>
KernelVariant grouped_variant_at() {
  using L = GroupedLayout<MODE, TT, OutTraits<OUT>::bytes>;
  return {reinterpret_cast<const void*>(&grouped_gemm_kernel<MODE, TT, BF16, OUT>), TT, L::STAGES,
          L::SMEM_BYTES, true, GROUPED_THREADS};
}

// The variants of one mode and operand type (a translation unit each): output
// in the operands' type OUT16 or in fp32, tiles up to tt = 64 or 256 wide.
template <int MODE, bool BF16, int OUT16>
KernelVariant grouped_variant_of(int out_kind, int tt) {
  if constexpr (MODE != GROUPED_DW) {
    if (tt == 64)
      return out_kind == OUT_F32 ? grouped_variant_at<MODE, 64, BF16, OUT_F32>()
                                 : grouped_variant_at<MODE, 64, BF16, OUT16>();
  }
  return out_kind == OUT_F32 ? grouped_variant_at<MODE, 256, BF16, OUT_F32>()
                             : grouped_variant_at<MODE, 256, BF16, OUT16>();
}

}  // namespace sptg
