// w4_tile_gemm.cuh -- products of 9 to 64 rows with 4-bit weights and group
// scales, on the fifth-generation tensor cores.
//
// The operator is w4_gemm.cuh's. Past 8 rows the warp-wide instruction of that
// kernel runs out of rate (1024 multiply-adds a cycle and SM: 56 us for the bare
// products of 64 rows with 32768 x 8192; such a kernel took 121 us), so the
// weights are widened once, into tensor memory, and one tcgen05 instruction
// multiplies 128 rows of them with all rows of x (swap-AB: the weights' rows are
// the instruction's M side, NTOK = 16, 32 or 64 rows of x its N side). Widened
// into shared memory instead, they are written and read there once each, four
// bytes a weight: 16 rows through 32768 x 8192 took 77 us, whatever else was
// changed.
//
// A CTA takes up to 128 rows of weights and a range of K (shared in a cluster,
// as in w4_gemm.cuh). Roles:
//
//   16 warps widen, in two groups that take the stages in turn (8 in one group
//            where registers are short): a lane turns 64 bytes of codes of its
//            row (128 of a stage's 256 columns) into its lane of the operand
//   4 warps  (8 past 16 rows of x) sums: a lane owns a row of weights; for each
//            group it reads the group's sums from tensor memory, multiplies them
//            by its scale and adds them to its own, in 32 bits
//   4 warps  widen a stage's x where it is 8-bit, ahead of the others (the fence
//            between their writes and the MMAs' reads is slow)
//   2 warps  producers of the two rings, codes and x, by tensor copy
//   1 warp   MMA issuer: a stage's 16 steps of 16 columns, one accumulator a
//            group
//
// Hand-overs are what a stage costs besides its work, so there are few: the
// issuer waits once for a stage's operands and once for its accumulators, issues
// the stage's MMAs without a branch and commits once, on a barrier that the
// widening warps (their operand is free), the producer of x (its stage is) and
// the sums (theirs are ready) all wait on. Two operands, and two sets of
// accumulators where they fit, alternate from stage to stage. A stage of codes
// leaves its ring when the codes have been written into the operand; x
// stays in its own until it has been multiplied. There is one issuer, in the order
// of the stages: a barrier that is waited on by its parity may then not run a whole
// turn ahead of any warp that waits on it (two issuers in turn would allow that).
//
// Measured (bf16, groups of 128): 16, 32 and 64 rows through 32768 x 8192 48.5,
// 54.3 and 63.9 us (the codes alone are 20 us at 6788 GB/s), through 8192 x 8192 16.4,
// 18.1 and 20.7 us; 16 int8 rows 15.8 us; 61 rows through 5001 x 4128 in groups of 32
// 19.5 us. More rows take a pass for each 64: 256, 1024 and 4096 rows through 8192 x
// 8192 62, 217 and 837 us (657 TFLOP/s). Scales and zero points read a lane's groups
// at a time, where alignment allows it, are worth most in small groups: 16 rows
// through 8192 x 8192 in groups of 32 with zero points went from 25.5 to 17.2 us
// (18.0 now).
// Not memory-bound (2.9 TB/s with 16 rows): a stage takes some 1200 cycles, of which
// the widening (11 to 13 instructions for 8 codes and lane, most of them on the
// integer pipe: 62 % of its cycles, 59 % of the issue slots) and the chain widen,
// hand over, 16 MMAs (some 500 cycles to issue), commit take about the same. The
// tensor pipe is busy 9 % (16 rows) to 25 % (64 rows) of the time. A third operand
// (51.5 to 50.6 us) and sleeping instead of polling (no difference) were not kept.
//
// Exactness: a widened weight is the integer code - zero point, |.| <= 15, in
// the 16-bit type of the product; products are exact, sums are kept in 32 bits,
// and the group's scale multiplies the group's 32-bit sum. Y is rounded once.
// (Scaling the widened weights instead would round each of them.)
#pragma once

#include "w4_gemm.cuh"

namespace sptg {

constexpr int W4T_MAX_ROWS = 128;
// Warps that widen the weights: 16, but 8 where other warps leave them too few
// registers (32 rows and more of 8-bit x). 64 rows of bf16 through 32768 x 8192:
// 64.4 us with 16 and 69.5 us with 8.
__host__ __device__ constexpr int w4t_widen(int xk, int ntok) {
  return ntok > 16 && xk >= W4_S8 ? 8 : 16;
}
// warps that widen x, where it is 8-bit
__host__ __device__ constexpr int w4t_widen_x(int xk) { return xk >= W4_S8 ? 4 : 0; }
// Stages of the ring of codes. Four at least: with an odd number a place in the
// ring goes from one group of widening warps to the other, and a group may wait
// for its next turn there only when the copy of the turn between has landed, or
// that turn's parity would be taken for its own. A group that comes to a stage
// knows that the one four before it has been multiplied.
constexpr int W4T_MIN_STAGES = 4;
constexpr int W4T_MAX_STAGES = 10;
// Warps for the sums: 8 share 32 rows of x and more (32 rows of binary16 through
// 32768 x 8192: 52.1 us against 57.7 us with 4).
__host__ __device__ constexpr int w4t_sum_warps(int ntok) { return ntok >= 32 ? 8 : 4; }
__host__ __device__ constexpr int w4t_threads(int xk, int ntok) {
  return 32 * (w4t_widen(xk, ntok) + w4t_sum_warps(ntok) + w4t_widen_x(xk) + 3);
}

// Tensor memory: 256 columns of accumulators, one for each group of a stage and
// row of x, then two operands of 128 columns (256 values of K).
constexpr int W4T_ACC_COLS = 256;
__host__ __device__ constexpr int w4t_max_ntok(int group) { return group == 32 ? 32 : 64; }

// Shared memory: the ring of codes, the ring of x (in 16 bits, and as copied
// where that is 8 bits), the barriers. The partial sums reuse the front.
__host__ __device__ constexpr int w4t_code_stage(int rows) { return rows * (W4_STAGE_K / 2); }
__host__ __device__ constexpr int w4t_x_bytes(int ntok) { return ntok * W4_STAGE_K * 2; }
__host__ __device__ constexpr int w4t_x_stage(int xk, int ntok) {
  return w4t_x_bytes(ntok) + (xk >= W4_S8 ? ntok * W4_STAGE_K : 0);
}
constexpr int W4T_MAX_X_STAGES = 4;
constexpr int W4T_BARS = 2 * W4T_MAX_STAGES + 2 * W4T_MAX_X_STAGES + 4 + 2 + 2 + 1;
__host__ __device__ constexpr int w4t_bars_at(int xk, int ntok, int rows, int stages, int x_stages) {
  const int rings = stages * w4t_code_stage(rows) + x_stages * w4t_x_stage(xk, ntok);
  const int red = ntok * (W4T_MAX_ROWS + 4) * 4;
  return rings > red ? rings : red;
}
__host__ __device__ constexpr int w4t_smem(int xk, int ntok, int rows, int stages, int x_stages) {
  return w4t_bars_at(xk, ntok, rows, stages, x_stages) + W4T_BARS * 8 + 16 + 1024;
}

// stages of x in their ring
__host__ __device__ constexpr int w4t_x_stages(int ntok) { return ntok == 64 ? 3 : W4T_MAX_X_STAGES; }
constexpr bool w4t_fits(int xk, int ntok) {
  return w4t_smem(xk, ntok, W4T_MAX_ROWS, W4T_MIN_STAGES, w4t_x_stages(ntok)) <= 232448;
}
static_assert(w4t_fits(W4_BF16, 64) && w4t_fits(W4_S8, 64) && w4t_fits(W4_BF16, 32) &&
                  w4t_fits(W4_S8, 32) && w4t_fits(W4_BF16, 16) && w4t_fits(W4_S8, 16),
              "the shortest ring of codes does not fit");

// The eight codes of a word, less the zero point (exact), as four columns of the
// operand: a mask and an exponent's bits make numbers of the codes of a word two
// at a time. z2, z2h: (-)(bias + zero point), what to take off in either half.
//
// 16-bit x is multiplied as copied, so the columns are in order: a byte
// permutation first brings two neighbours to the low byte of either half.
// bfloat16 has room for a code in the low four bits only (128 + code; the odd
// ones come from the word moved down four bits); binary16 takes the odd ones
// where they are, as 1024 + 16 code, and a multiply-add makes (1, 1 / 16) of them.
//
// 8-bit x is rewritten on its way anyway, in the order that a word's halves give
// without permutations: (0, 4) (1, 5) (2, 6) (3, 7). (16 rows of int8 through
// 8192 x 8192: 14.8 us against 15.9 with the codes put in order.)
template <int XK>
__device__ __forceinline__ void widen_word(const W4Params& p, uint32_t w, uint32_t z2, uint32_t z2h,
                                           uint32_t* o) {
  auto sub = [](uint32_t v, uint32_t z) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&z));
    return *reinterpret_cast<const uint32_t*>(&d);
  };
  auto fma = [](uint32_t v, uint32_t f, uint32_t z) {
    const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&f),
                              *reinterpret_cast<const __half2*>(&z));
    return *reinterpret_cast<const uint32_t*>(&d);
  };
  if constexpr (XK >= W4_S8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[2 * i] = sub(pick(w >> (8 * i), p.mask_lo, p.magic), z2);
      o[2 * i + 1] = fma(pick(w >> (8 * i), p.mask_hi, p.magic), 0x2c002c00u, z2h);
    }
  } else {
    const uint32_t odd = XK == W4_BF16 ? w >> 4 : w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = pick(__byte_perm(w, odd, (4 + i) << 8 | i), p.mask_tile, p.magic);
      if constexpr (XK == W4_BF16) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         *reinterpret_cast<const __nv_bfloat162*>(&z2));
        o[i] = *reinterpret_cast<const uint32_t*>(&d);
      } else {
        o[i] = fma(v, 0x2c003c00u, z2);
      }
    }
  }
}

template <int XK, int NTOK, int G>
__global__ void __launch_bounds__(w4t_threads(XK, NTOK), 1)
    w4_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const W4Params p) {
  constexpr bool BF = XK == W4_BF16;
  constexpr bool X8 = XK >= W4_S8;
  constexpr int GROUPS = W4_STAGE_K / G;
  constexpr uint32_t IDESC = idesc_f16_f32acc(BF, 128, NTOK);
  constexpr int SUMS = w4t_sum_warps(NTOK);
  constexpr int WIDEN = w4t_widen(XK, NTOK);
  constexpr int WIDEN_X = WIDEN + SUMS, PRODUCER = WIDEN_X + w4t_widen_x(XK);  // first warps of the roles
  constexpr int X_PRODUCER = PRODUCER + 1, ISSUER = PRODUCER + 2;
  constexpr int COLS = NTOK * 4 / SUMS;  // rows of x a sums warp holds
  constexpr int ACC_SET = GROUPS * NTOK;  // columns of a stage's accumulators
  constexpr int SETS = 2 * ACC_SET <= W4T_ACC_COLS ? 2 : 1;
  static_assert(ACC_SET <= W4T_ACC_COLS, "accumulators exceed their part of tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  const int S = p.stages, SX = p.segment, R = p.rows;
  const uint32_t ring = sbase;
  const uint32_t x_ring = ring + S * w4t_code_stage(R);
  constexpr int X_STAGE = w4t_x_stage(XK, NTOK);
  constexpr int OFF_RAW = w4t_x_bytes(NTOK);  // in a stage of x: x as copied, if 8-bit
  const int off_bars = w4t_bars_at(XK, NTOK, R, S, SX);
  const uint32_t bar0 = sbase + off_bars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };  // codes
  auto empty_bar = [&](int s) { return bar0 + 8u * (W4T_MAX_STAGES + s); };
  const uint32_t bar1 = bar0 + 8u * (2 * W4T_MAX_STAGES);
  auto xfull_bar = [&](int s) { return bar1 + 8u * s; };
  auto xready_bar = [&](int s) { return bar1 + 8u * (W4T_MAX_X_STAGES + s); };  // widened
  const uint32_t bar2 = bar1 + 8u * (2 * W4T_MAX_X_STAGES);
  auto done_bar = [&](int it) { return bar2 + 8u * (it & 3); };         // stage multiplied
  auto done_parity = [](int it) { return static_cast<uint32_t>(it >> 2) & 1u; };
  auto ready_bar = [&](int it) { return bar2 + 8u * (4 + (it & 1)); };  // widened
  auto tempty_bar = [&](int it) { return bar2 + 8u * (6 + it % SETS); };  // sums read
  auto pair_parity = [](int it) { return static_cast<uint32_t>(it >> 1) & 1u; };
  const uint32_t drain_bar = bar0 + 8u * (W4T_BARS - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + off_bars + W4T_BARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + off_bars + W4T_BARS * 8 + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * R;
  const int m0 = p.m_first + static_cast<int>(blockIdx.y) * NTOK;
  const int KS = (p.K + W4_STAGE_K - 1) / W4_STAGE_K;
  const int ks0 = static_cast<int>(static_cast<int64_t>(KS) * rank / p.splits);
  const int ks1 = static_cast<int>(static_cast<int64_t>(KS) * (rank + 1) / p.splits);
  const int stages = ks1 - ks0;
  const int KG = p.K / G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 8);  // a group of widening warps
    }
    for (int s = 0; s < SX; ++s) {
      mbar_init(xfull_bar(s), 1);
      if (X8) mbar_init(xready_bar(s), w4t_widen_x(XK));
    }
    for (int i = 0; i < 4; ++i) mbar_init(done_bar(i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(ready_bar(i), 8);
      mbar_init(tempty_bar(i), SUMS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensor_map(&tmW);
    prefetch_tensor_map(&tmX);
  }
  if (warp == ISSUER) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  const WaitCtl ctl{p.timeout_ns, p.error_word, abort_flag};
  // the whole warp waits together
  auto wait = [&](uint32_t bar, uint32_t parity, unsigned int site) {
    return __all_sync(0xffffffffu, wait_bounded_lazy(bar, parity, ctl, site));
  };
  float acc[COLS];  // sums warps: this lane's row of weights
#pragma unroll
  for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;

  if (warp < WIDEN) {
    // ---------------------------------------------------------------- widen
    // Thread: row r (= its lane of tensor memory), columns 128 c ... + 127 of a
    // stage.
    constexpr int GRPS = WIDEN / 8;
    const int group = warp >> 3;
    const int r = threadIdx.x & 127, c = (threadIdx.x >> 7) & 1;
    const bool works = r < R;
    const uint8_t* zp = p.zeros ? p.zeros + static_cast<int64_t>(min(n0 + r, p.N - 1)) * KG : nullptr;
    constexpr int ZS = 128 / G;  // zero points of a lane's columns
    uint32_t next_z[ZS];
#pragma unroll
    for (int i = 0; i < ZS; ++i) next_z[i] = 8u;
    auto load_zeros = [&](int ks) {
      if (!zp) return;
      const int at = (ks * W4_STAGE_K + 128 * c) / G;
      if (ZS == 4 && p.wide) {
        next_z[0] = *reinterpret_cast<const uint32_t*>(zp + at);
      } else if (ZS == 2 && p.wide) {
        next_z[0] = *reinterpret_cast<const uint16_t*>(zp + at);
      } else {
#pragma unroll
        for (int i = 0; i < ZS; ++i) next_z[i] = zp[min(at + i, KG - 1)];
      }
    };
    load_zeros(min(ks0 + group, ks1 - 1));
    // places that do not change from stage to stage: this lane's row of codes
    // (128-byte aligned; piece i lies at place i ^ (r & 7)) and its columns of
    // the operand
    const uint32_t code0 = static_cast<uint32_t>(r * 128 + (((4 * c) ^ (r & 7)) << 4));
    const uint32_t dst0 = tmem_base + W4T_ACC_COLS + 64 * c + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    int s = group;
    uint32_t phase = 0;
    for (int it = group; it < stages; it += GRPS) {
      uint32_t z[ZS];
#pragma unroll
      for (int i = 0; i < ZS; ++i) {
        asm volatile("" : "+r"(next_z[i]));  // no use of the loads before this
        z[i] = (ZS > 1 && p.wide && zp ? next_z[0] >> (8 * i) : next_z[i]) & 15u;
      }
      load_zeros(min(ks0 + it + GRPS, ks1 - 1));
      if (!wait(full_bar(s), phase, WAIT_MMA_FULL)) break;
      const uint32_t st = ring + s * w4t_code_stage(R);
      uint4 code[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        code[i] = works ? lds128(st + (code0 ^ static_cast<uint32_t>(i << 4))) : make_uint4(0, 0, 0, 0);
      // the operand's last multiplication, two stages ago, has ended
      if (it >= 2) {
        if (!wait(done_bar(it - 2), done_parity(it - 2), WAIT_PRODUCER_EMPTY)) break;
        tc_fence_after();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t zi = z[i * ZS / 4];
        // 128 + z; 1024 + z and -(64 + z); -(1024 + z) beside -(64 + z)
        const uint32_t z2 = BF ? (0x4300u | zi) * 0x00010001u
                            : X8 ? (0x6400u | zi) * 0x00010001u : 0xd400e400u | zi | zi << 20;
        const uint32_t z2h = (0xd400u | zi << 4) * 0x00010001u;
        const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        uint32_t o[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) widen_word<XK>(p, w[k], z2, z2h, o + 4 * k);
        tmem_st_32x32b_x16(dst0 + (it & 1) * 128 + 16 * i, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      // The stage of codes goes back only here, when its codes have been used: an
      // arrival right behind the loads left the loads themselves free to run after
      // the wait above, when the next copy had overwritten the codes (17 stages in
      // groups of 32, whose slow sums make that wait long: every call had wrong
      // groups). Nothing is lost by it: eight to ten stages are in flight.
      if (lane == 0) {
        mbar_arrive(empty_bar(s));
        mbar_arrive(ready_bar(it));
      }
      s += GRPS;
      if (s >= S) {
        s -= S;
        phase ^= 1u;
      }
    }
  } else if (warp < WIDEN_X) {
    // ----------------------------------------------------------------- sums
    const int q = warp & 3;
    const int r = 32 * q + lane;
    const int col0 = warp >= WIDEN + 4 ? COLS : 0;
    const uint16_t* sp = p.scales + static_cast<int64_t>(min(n0 + r, p.N - 1)) * KG;
    // A stage's scales, a stage ahead; where alignment allows it in one load, two
    // to a register. Groups past K have no sums but zeros. (No non-coherent loads
    // here and above, as in w4_gemm.cuh.)
    uint32_t next_s[GROUPS];
    auto load_scales = [&](int ks) {
      if (p.wide) {
        const uint16_t* at = sp + ks * GROUPS;
        if constexpr (GROUPS == 8)
          asm volatile("ld.global.L2::128B.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(next_s[0]), "=r"(next_s[1]), "=r"(next_s[2]), "=r"(next_s[3])
                       : "l"(at)
                       : "memory");
        else if constexpr (GROUPS == 4)
          asm volatile("ld.global.L2::128B.v2.b32 {%0, %1}, [%2];"
                       : "=r"(next_s[0]), "=r"(next_s[1])
                       : "l"(at)
                       : "memory");
        else
          asm volatile("ld.global.L2::128B.b32 %0, [%1];" : "=r"(next_s[0]) : "l"(at) : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
          asm volatile("ld.global.L2::128B.u16 %0, [%1];"
                       : "=r"(next_s[i])
                       : "l"(sp + min(ks * GROUPS + i, KG - 1))
                       : "memory");
      }
    };
    load_scales(ks0);
    for (int it = 0; it < stages; ++it) {
      float sc[GROUPS];
      const bool bf = BF || (XK != W4_F16 && p.out_bf16);
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) asm volatile("" : "+r"(next_s[i]));  // no use before this
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        const uint32_t h = p.wide ? next_s[i >> 1] >> (16 * (i & 1)) : next_s[i];
        sc[i] = bf ? __uint_as_float(h << 16)
                   : __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
      }
      load_scales(min(ks0 + it + 1, ks1 - 1));
      if (!wait(done_bar(it), done_parity(it), WAIT_EPI_TMEM_FULL)) break;
      tc_fence_after();
      const uint32_t t_acc =
          tmem_base + it % SETS * ACC_SET + col0 + (static_cast<uint32_t>(32 * q) << 16);
      // 16 sums at a time: with 32 in flight the registers would not do
#pragma unroll
      for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int h = 0; h < COLS; h += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(t_acc + g * NTOK + h, v);
          tmem_wait_ld_regs16(v);
          if (g == GROUPS - 1 && h == COLS - 16) {  // all have been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(it));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[h + i] = fmaf(sc[g], __uint_as_float(v[i]), acc[h + i]);
        }
    }
  } else if (warp < PRODUCER) {
    // -------------------------------------------------------------- widen x
    if constexpr (X8) {
      // Pieces of 8 columns: this lane's first (row pw of x, piece lane of a
      // stage's 32; then 4 rows on, whose place under the swizzle differs in
      // one bit).
      const int pw = warp - WIDEN_X;
      const uint32_t piece0 = static_cast<uint32_t>((lane >> 3) * (NTOK * 128) + pw * 128 +
                                                    (((lane & 7) ^ pw) << 4));
      const uint32_t raw0 = static_cast<uint32_t>(OFF_RAW + pw * W4_STAGE_K + lane * 8);
      int sx = 0;
      uint32_t phase = 0;
      for (int it = 0; it < stages; ++it) {
        if (!wait(xfull_bar(sx), phase, WAIT_MMA_FULL)) break;
        const uint32_t st = x_ring + sx * X_STAGE;
#pragma unroll
        for (int m = 0; m < NTOK; m += 4) {
          const uint4 v = pair_x<XK>(make_uint4(lds32(st + raw0 + m * W4_STAGE_K),
                                                lds32(st + raw0 + m * W4_STAGE_K + 4), 0, 0));
          // (the pairs (0,4) (2,6) (1,5) (3,7))
          sts128((st + piece0 + m * 128) ^ ((m & 4) << 4), make_uint4(v.x, v.z, v.y, v.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(xready_bar(sx));
        if (++sx == SX) {
          sx = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == PRODUCER || warp == X_PRODUCER) {
    // ------------------------------------------------------------ producers
    const bool leader = elect_one_sync();
    const bool of_x = warp == X_PRODUCER;
    const uint64_t pol =
        of_x || gridDim.y > 1 ? policy_evict_last() : policy_evict_first();
    const int depth = of_x ? SX : S;
    auto full = [&](int s) { return of_x ? xfull_bar(s) : full_bar(s); };
    int issued = 0;
    bool ok = true;
    int s = 0;
    uint32_t phase = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
      const int it = ks - ks0;
      if (!of_x)
        ok = wait(empty_bar(s), phase ^ 1u, WAIT_PRODUCER_EMPTY);
      else if (it >= SX)
        ok = wait(done_bar(it - SX), done_parity(it - SX), WAIT_PRODUCER_EMPTY);
      if (!ok) break;
      if (leader) {
        if (!of_x) {
          mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(w4t_code_stage(R)));
          tma_load_2d(ring + s * w4t_code_stage(R), &tmW, full_bar(s), ks * (W4_STAGE_K / 2), n0, pol);
        } else {
          const uint32_t st = x_ring + s * X_STAGE;
          mbar_arrive_expect_tx(xfull_bar(s), X8 ? NTOK * W4_STAGE_K : w4t_x_bytes(NTOK));
          if constexpr (X8) {
            tma_load_2d(st + OFF_RAW, &tmX, xfull_bar(s), ks * W4_STAGE_K, m0, pol);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tma_load_2d(st + c * (NTOK * 128), &tmX, xfull_bar(s), ks * W4_STAGE_K + 64 * c, m0, pol);
          }
        }
      }
      ++issued;
      if (++s == depth) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (!of_x) grid_launch_dependents();
    if (!ok) {
      // let every copy already issued land before the CTA can exit
      for (int i = max(0, issued - depth); i < issued; ++i) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(full(i % depth), static_cast<uint32_t>(i / depth) & 1u) &&
               global_timer_ns() - t0 < ctl.timeout_ns) {
        }
      }
    }
  } else {
    // ----------------------------------------------------------- MMA issuer
    const bool leader = elect_one_sync();
    int sx = 0;
    uint32_t x_phase = 0;
    for (int it = 0; it < stages; ++it) {
      if (!wait(X8 ? xready_bar(sx) : xfull_bar(sx), x_phase, WAIT_MMA_FULL)) break;
      if (!wait(ready_bar(it), pair_parity(it), WAIT_MMA_FULL)) break;
      if (it >= SETS &&
          !wait(tempty_bar(it), (static_cast<uint32_t>(it / SETS) & 1u) ^ 1u, WAIT_MMA_TMEM_EMPTY))
        break;
      tc_fence_after();
      const uint32_t at = tmem_base + W4T_ACC_COLS + (it & 1) * 128;
      const uint64_t xd = sdesc_k_major_sw128(x_ring + sx * X_STAGE);
      const uint32_t d = tmem_base + it % SETS * ACC_SET;
      if (leader) {
        // steps of 16 columns (8 of tensor memory), G / 16 a group
#pragma unroll
        for (int k = 0; k < W4_STAGE_K / 16; ++k)
          mma_f16_ts(d + k / (G / 16) * NTOK, at + 8 * k,
                     xd + static_cast<uint64_t>((k >> 2) * (NTOK * 128) >> 4) + 2 * (k & 3), IDESC,
                  k % (G / 16) == 0 ? 0u : 1u);
        mma_commit(done_bar(it));
      }
      __syncwarp();
      if (++sx == SX) {
        sx = 0;
        x_phase ^= 1u;
      }
    }
    if (leader) mma_commit(drain_bar);
    __syncwarp();
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(drain_bar, 0) && global_timer_ns() - t0 < ctl.timeout_ns) {
    }
  }
  // Every MMA and copy has completed: the partial sums take the front of
  // shared memory.
  tc_fence_before();
  __syncthreads();
  if (warp == ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  const int pitch = W4T_MAX_ROWS + 4;
  if (warp >= WIDEN && warp < WIDEN_X) {
    const int col0 = warp >= WIDEN + 4 ? COLS : 0;
    float* red = reinterpret_cast<float*>(smem) + col0 * pitch + 32 * (warp & 3) + lane;
#pragma unroll
    for (int i = 0; i < COLS; ++i) red[i * pitch] = acc[i];
  }
  __syncwarp();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each CTA of the cluster adds up its share of the rows of weights, over
  // the CTAs in order.
  const int rows = R / p.splits;
  const int live_m = min(NTOK, p.M - m0);
  for (int i = threadIdx.x; i < rows * live_m; i += w4t_threads(XK, NTOK)) {
    const int m = i / rows, r = rank * rows + i % rows;
    const uint32_t at = sbase + static_cast<uint32_t>((m * pitch + r) * 4);
    float v = 0.0f;
    for (int c = 0; c < p.splits; ++c) {
      float x;
      if (p.splits > 1)
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(map_to_cta(at, static_cast<uint32_t>(c)))
                     : "memory");
      else
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
      v += x;
    }
    if (p.x_scales) v *= p.x_scales[m0 + m];
    if (n0 + r < p.N) {
      if (p.out_bf16)
        store_out<OUT_BF16>(p.out, static_cast<int64_t>(m0 + m) * p.ldo + n0 + r, v);
      else
        store_out<OUT_F16>(p.out, static_cast<int64_t>(m0 + m) * p.ldo + n0 + r, v);
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// The variants of one kind of x (part of its translation unit).
template <int XK>
const void* w4_tile_kernel_of(int ntok, int group) {
#define SPTG_W4T_CASE(NTOK_, G_) \
  if (ntok == NTOK_ && group == G_) return reinterpret_cast<const void*>(&w4_tile_kernel<XK, NTOK_, G_>)
  SPTG_W4T_CASE(16, 32);
  SPTG_W4T_CASE(16, 64);
  SPTG_W4T_CASE(16, 128);
  SPTG_W4T_CASE(32, 32);
  SPTG_W4T_CASE(32, 64);
  SPTG_W4T_CASE(32, 128);
  SPTG_W4T_CASE(64, 64);
  SPTG_W4T_CASE(64, 128);
#undef SPTG_W4T_CASE
  return nullptr;
}

}  // namespace sptg
