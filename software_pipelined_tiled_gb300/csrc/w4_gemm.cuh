// w4_gemm.cuh -- products of up to 8 rows with 4-bit weights and group scales.
//
//   Y[m, n] = xs[m] * sum_g s[n, g] * sum_{k in group g} x[m, k] * (w[n, k] - z[n, g])
//
// w: 4-bit codes 0 ... 15, two to a byte along K (the even column in the low
// half); s: a 16-bit scale for each row of weights and group of G = 32, 64 or
// 128 columns; z: a zero point 0 ... 15 for each group, or 8 everywhere; x: 16
// bits, or 8 bits (int8, e4m3) with a 32-bit scale xs for each row.
//
// Exactness: a code less its zero point is an integer of at most 15, exact in the
// 16-bit type of the product (8-bit x is exact in binary16). The products are
// exact, the sums are kept in 32 bits for each group, and the group's scale
// multiplies the group's sum as it is added to the running sum in 32 bits. The
// only rounding to 16 bits is that of Y. (Taking the zero points out of the
// groups' sums instead, sum x (w - z) = sum x w - z sum x, with codes that are
// masked only, forms sums 10 to 30 times as large, whose rounding does not cancel,
// and turns an infinity in x into NaN. It saved 8 instructions for 16 x 32 codes
// and needed the sums of x: one binary16 row through 32768 x 8192 36.2 us against
// 38.0, one bf16 row 34.6 against 34.7, 8 bf16 rows 45.9 against 42.5.)
//
// Memory-bound: N * K / 2 bytes of codes, each read once. A CTA takes a block of
// rows of weights and a range of K (the whole, or a share of it in a cluster of
// 2, 4 or 8 CTAs, whose partial sums meet through distributed shared memory in
// CTA order: no atomics, the result does not depend on timing). It keeps its
// range of x in shared memory, in the order and type the products use; where x
// is too large for that, it goes through K in segments. Each warp streams the
// codes of its own 16 rows through a ring of its own with the tensor-copy engine
// (stages of 256 columns: 128 bytes a row, 128-byte swizzled) and refills a stage
// when it has read it, so that no warp ever waits for another inside a segment.
//
// Measured: one bf16 row through 4096 x 4096, 8192 x 8192, 16384 x 4096 and
// 32768 x 8192 in groups of 128 5.8, 13.6, 12.7 and 34.7 us back to back, 8 rows
// 7.0, 15.0, 13.4 and 42.5 us; one int8 row through 8192 x 8192 13.9 us, 8 16.5. One
// binary16 row through 32768 x 8192, groups of 64 with zero points, 38.0 us
// (3.9 TB/s; the floor at 6788 GB/s is 21.7 us). The copies alone take 23.4 us;
// what remains is bound by the issue of the instructions that make operands of the
// codes (61 % of the slots, 44 % of the integer pipe). A ring shared by the CTA, x
// travelling in its stages, needed two CTA-wide barriers a stage and took 46 us,
// whatever was taken out of the arithmetic.
//
// The multiply is the warp-wide 16 x 8 x 16 instruction, whose operands live
// in registers: codes are spread in registers and never stored, and with up to
// 8 rows of x the instruction's rate (1024 multiply-adds a cycle and SM) is far
// above what memory delivers. More rows go to w4_tile_gemm.cuh.
//
// Order within K: the products' sum does not depend on which columns share an
// instruction, as long as both operands agree. Lane (g, t) = (lane / 4, lane
// mod 4) of a warp reads one 32-bit word of codes -- columns 8t ... 8t + 7 of
// a unit of 32 columns -- for its rows g and g + 8. Masking the word after
// shifts leaves the column pairs (0, 4), (1, 5), (2, 6), (3, 7), which feed two
// instructions; x's eight values are paired the same way when x is stored.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sptg {

// Rows of x as they lie in memory. 16-bit x multiplies in its own type, 8-bit
// x in binary16.
enum W4X : int { W4_BF16 = 0, W4_F16 = 1, W4_S8 = 2, W4_E4M3 = 3 };

constexpr int W4_STAGE_K = 256;   // columns per ring stage
constexpr int W4_UNITS = 8;       // units of 32 columns in a stage
constexpr int W4_MAX_STAGES = 8;  // of a warp's ring
constexpr int W4_X_ROWS = 8;      // rows of x: the instruction's N side
constexpr int W4_WARP_ROWS = 16;  // rows of weights of a warp: its M side
// Two warps share rows of weights, each with half of a segment's K: with one
// wave of CTAs 14 warps to an SM would otherwise have to hide the latency of
// their own instructions.
constexpr int W4_KW = 2;
// Up to 14 warps to a CTA, two CTAs to an SM with 72 registers a thread.
constexpr int W4_MAX_WARPS = 14;
constexpr int W4_CTAS_PER_SM = 2;
constexpr int W4_MAX_ROWS = W4_WARP_ROWS * W4_MAX_WARPS / W4_KW;

struct W4Params {
  int M, N, K;
  int m_first;             // tile kernel: first row of x of this launch
  const void* x;           // M rows of K, ldx elements apart
  int64_t ldx;
  int rows;                // rows of weights per CTA, a multiple of 16
  int stages;              // depth of each warp's ring
  int splits;              // CTAs of the cluster, sharing K
  int segment;             // stages of K whose x is held at a time (tile kernel: depth of
                           // the ring of x)
  const uint16_t* scales;  // N x K / G
  const uint8_t* zeros;    // N x K / G, or null (8)
  const float* x_scales;   // M, or null (1)
  uint16_t* out;           // M rows of N, ldo apart
  int64_t ldo;
  int out_bf16;            // type of scales and out: bfloat16, else binary16
  int wide;                // scales (and zeros) read a lane's groups at a time
  uint32_t mask_lo, mask_hi, magic;  // of spread_codes
  uint32_t mask_tile;                // of widen_word
  unsigned int* error_word;
  uint64_t timeout_ns;
};

__host__ __device__ constexpr int w4_x_bytes(int xk) { return xk >= W4_S8 ? 1 : 2; }

// Shared memory of a CTA, in this order: the rings, x (16 bits), the scales, the
// barriers. The partial sums reuse the front.
struct W4Layout {
  int warps, ring, x, table, bars, total;
};
__host__ __device__ constexpr int w4_red_pitch(int rows) { return rows + 4; }
__host__ __device__ constexpr W4Layout w4_layout(int group, int rows, int stages, int segment,
                                                 int live_m) {
  W4Layout l{};
  l.warps = rows / W4_WARP_ROWS * W4_KW;
  l.ring = 0;
  l.x = l.warps * stages * W4_WARP_ROWS * (W4_STAGE_K / 2);
  l.table = l.x + segment * live_m * W4_STAGE_K * 2;
  l.bars = l.table + l.warps * W4_WARP_ROWS * (W4_STAGE_K / group) * 8;
  // (the partial sums of all warps take the place of everything before)
  const int red = W4_KW * W4_X_ROWS * w4_red_pitch(rows) * 4;
  if (l.bars < red) l.bars = (red + 15) & ~15;
  l.total = l.bars + W4_MAX_WARPS * W4_MAX_STAGES * 8 + 16;
  return l;
}

// d = a b + (first ? 0 : d); a literal zero takes no registers
template <bool BF>
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1, bool first) {
  const float c[4] = {first ? 0.0f : d[0], first ? 0.0f : d[1], first ? 0.0f : d[2],
                      first ? 0.0f : d[3]};
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

// Loads from shared memory. The memory clobber keeps them between the wait for
// what they read and the hand-over that lets it be overwritten; `volatile` alone
// does not.
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ float2 lds64f(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// b = 1024 + 128 + a in each half, to a
__device__ __forceinline__ uint32_t unbias2(uint32_t b) {
  constexpr uint32_t BIAS = 0x64806480u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&BIAS));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// (w & mask) | magic in one instruction
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
  return r;
}

// The zero point of a group as spread_codes takes it, in both halves: 128 + z in
// bfloat16, 1024 + z in binary16.
template <bool BF>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  return ((BF ? 0x4300u : 0x6400u) | z) * 0x00010001u;
}
// binary16: -(64 + z) beside it, for the codes in bits 4-7
__device__ __forceinline__ uint32_t zero_pair_high(uint32_t z2) {
  return pick(z2 << 4, 0x00f000f0u, 0xd400d400u);
}

// The eight codes of a word, less the zero point, as column pairs: (0,4), (2,6)
// in `a`, (1,5), (3,7) in `b`. A mask and an exponent's bits make numbers of the
// codes of a word two at a time (a published method for 4-bit weights; the
// constants follow from the two formats), and one subtraction (exact) takes the zero point
// and the exponent's own value off both. Binary16 takes the codes of bits 4-7
// where they are, as 1024 + 16 code, and a multiply-add brings them down;
// bfloat16 has room for a code in the low four bits only: three shifts.
template <bool BF>
__device__ __forceinline__ void spread_codes(const W4Params& p, uint32_t w, uint32_t z2,
                                             uint32_t z2h, uint32_t (&a)[2], uint32_t (&b)[2]) {
  if constexpr (BF) {
    auto sub = [&](uint32_t v) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                       *reinterpret_cast<const __nv_bfloat162*>(&z2));
      return *reinterpret_cast<const uint32_t*>(&d);
    };
    a[0] = sub(pick(w, p.mask_lo, p.magic));
    b[0] = sub(pick(w >> 4, p.mask_lo, p.magic));
    a[1] = sub(pick(w >> 8, p.mask_lo, p.magic));
    b[1] = sub(pick(w >> 12, p.mask_lo, p.magic));
  } else {
    constexpr uint32_t SIXTEENTH = 0x2c002c00u;
    const __half2 z = *reinterpret_cast<const __half2*>(&z2);
    const __half2 zh = *reinterpret_cast<const __half2*>(&z2h);
    const __half2 f = *reinterpret_cast<const __half2*>(&SIXTEENTH);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = pick(w >> (8 * i), p.mask_lo, p.magic), hi = pick(w >> (8 * i), p.mask_hi, p.magic);
      const __half2 dl = __hsub2(*reinterpret_cast<const __half2*>(&lo), z);
      const __half2 dh = __hfma2(*reinterpret_cast<const __half2*>(&hi), f, zh);
      a[i] = *reinterpret_cast<const uint32_t*>(&dl);
      b[i] = *reinterpret_cast<const uint32_t*>(&dh);
    }
  }
}

// One lane's eight values of x of one unit (8-bit: in v.x and v.y), from memory's order to the column
// pairs of spread_codes, in the type of the product.
template <int XK>
__device__ __forceinline__ uint4 pair_x(const uint4 v) {
  if constexpr (XK == W4_BF16 || XK == W4_F16) {
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x7632));
  } else {
    const uint32_t lo = __byte_perm(v.x, v.y, 0x5140);  // bytes 0, 4, 1, 5
    const uint32_t hi = __byte_perm(v.x, v.y, 0x7362);  // bytes 2, 6, 3, 7
    if constexpr (XK == W4_S8) {
      // a byte with its sign bit flipped is b + 128; under the exponent byte
      // 0x64 it is 1024 + b + 128 in binary16, and 1152 less leaves b
      constexpr uint32_t E = 0x64646464u;
      const uint32_t l = lo ^ 0x80808080u, h = hi ^ 0x80808080u;
      return make_uint4(unbias2(__byte_perm(l, E, 0x4140)), unbias2(__byte_perm(h, E, 0x4140)),
                        unbias2(__byte_perm(l, E, 0x4342)), unbias2(__byte_perm(h, E, 0x4342)));
    } else {
      const uint32_t q[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw r =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q[i]), __NV_E4M3);
        b[i] = static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
      }
      return make_uint4(b[0], b[2], b[1], b[3]);
    }
  }
}

template <int XK, int G>
__global__ void __launch_bounds__(32 * W4_MAX_WARPS, W4_CTAS_PER_SM)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const W4Params p) {
  constexpr bool BF = XK == W4_BF16;
  constexpr int XB = w4_x_bytes(XK);
  constexpr int KW = W4_KW, WR = W4_WARP_ROWS;
  constexpr int GROUPS = W4_STAGE_K / G;      // groups in a stage
  constexpr int UPG = G / 32;                 // units in a group
  constexpr int STAGE = WR * (W4_STAGE_K / 2);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = p.stages;
  const int R = p.rows;
  const W4Layout lay = w4_layout(G, R, S, p.segment, p.M);
  const uint32_t sbase = smem_addr(smem);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + lay.bars + W4_MAX_WARPS * W4_MAX_STAGES * 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % p.splits;  // = the CTA's rank in its cluster
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * R;
  const int rw = warp / KW, kw = warp % KW;  // block of rows, part of K
  const int row0 = n0 + WR * rw;
  const uint32_t ring = sbase + warp * S * STAGE;
  const uint32_t full0 = sbase + lay.bars + warp * (W4_MAX_STAGES * 8);
  // this CTA's stages of K, in segments; a warp's part of segment i is
  // [part_of(i, kw), part_of(i, kw + 1))
  const int KS = (p.K + W4_STAGE_K - 1) / W4_STAGE_K;
  const int ks0 = static_cast<int>(static_cast<int64_t>(KS) * rank / p.splits);
  const int ks1 = static_cast<int>(static_cast<int64_t>(KS) * (rank + 1) / p.splits);
  const int segments = (ks1 - ks0 + p.segment - 1) / p.segment;
  auto part_of = [&](int seg, int part) {
    const int a = ks0 + seg * p.segment, b = min(ks1, a + p.segment);
    return a + (b - a) * part / KW;
  };

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full0 + 8 * s, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefetch_tensor_map(&tmW);
  }
  __syncthreads();
  grid_dependency_wait();
  const WaitCtl ctl{p.timeout_ns, p.error_word, abort_flag};

  // The copies run ahead of the products through segments and stages.
  const bool leader = elect_one_sync();
  const uint64_t pol = policy_evict_first();  // codes are read once
  int issued = 0;
  int next_seg = 0;
  int next_ks = segments > 0 ? part_of(0, kw) : 0, next_end = segments > 0 ? part_of(0, kw + 1) : 0;
  auto issue_next = [&](int s) {
    while (next_ks >= next_end) {  // the next segment in which this warp has a part
      if (++next_seg >= segments) return;
      next_ks = part_of(next_seg, kw);
      next_end = part_of(next_seg, kw + 1);
    }
    if (leader) {
      mbar_arrive_expect_tx(full0 + 8 * s, STAGE);
      tma_load_2d(ring + s * STAGE, &tmW, full0 + 8 * s, next_ks * (W4_STAGE_K / 2), row0, pol);
    }
    ++next_ks;
    ++issued;
  };
  for (int s = 0; s < S; ++s) issue_next(s);

  // Scales and zero points. A lane fetches those of one row for PG groups of
  // a stage, a stage ahead, and then writes what the products use -- the
  // factor of a group's sum of products and that of its sum of x, in 32 bits --
  // into the warp's table of [group][row of the warp]. Rows past N read the
  // last row's. Where every row's scales fill whole stages and lie aligned
  // (p.wide), PG of them are one load; elsewhere one by one, with groups past
  // the end dropped.
  const int KG = p.K / G;
  constexpr int PG = GROUPS / 2;
  const int srow = min(row0 + (lane & 15), p.N - 1);
  const int sgroup = (lane >> 4) * PG;  // the lane's first group of a stage
  const uint16_t* my_scales = p.scales + static_cast<int64_t>(srow) * KG + sgroup;
  const uint8_t* my_zeros =
      p.zeros ? p.zeros + static_cast<int64_t>(srow) * KG + sgroup : nullptr;
  float2* table = reinterpret_cast<float2*>(smem + lay.table) + warp * (WR * GROUPS) + sgroup * WR +
                  (lane & 15);
  uint32_t next_s[(PG + 1) / 2], next_z[(PG + 3) / 4];  // as they lie in memory
  auto load_scales = [&](int ks) {
    const uint16_t* ps = my_scales + ks * GROUPS;
    const uint8_t* pz = my_zeros + ks * GROUPS;
    // (rows are far apart: a whole line of each is called into L2 at once. Not the
    // non-coherent path: the call before, which may have written them, can still
    // have been running when this kernel started)
    if (p.wide) {
      if constexpr (PG == 1)
        asm volatile("ld.global.L2::128B.u16 %0, [%1];" : "=r"(next_s[0]) : "l"(ps) : "memory");
      else if constexpr (PG == 2)
        asm volatile("ld.global.L2::128B.b32 %0, [%1];" : "=r"(next_s[0]) : "l"(ps) : "memory");
      else
        asm volatile("ld.global.L2::128B.v2.b32 {%0, %1}, [%2];"
                     : "=r"(next_s[0]), "=r"(next_s[PG / 2 - 1])
                     : "l"(ps)
                     : "memory");
      if (p.zeros) {
        if constexpr (PG == 1)
          asm volatile("ld.global.L2::128B.u8 %0, [%1];" : "=r"(next_z[0]) : "l"(pz) : "memory");
        else if constexpr (PG == 2)
          asm volatile("ld.global.L2::128B.u16 %0, [%1];" : "=r"(next_z[0]) : "l"(pz) : "memory");
        else
          asm volatile("ld.global.L2::128B.b32 %0, [%1];" : "=r"(next_z[0]) : "l"(pz) : "memory");
      }
    } else {
#pragma unroll
      for (int i = 0; i < (PG + 1) / 2; ++i) next_s[i] = 0;
#pragma unroll
      for (int i = 0; i < (PG + 3) / 4; ++i) next_z[i] = 0;
#pragma unroll
      for (int i = 0; i < PG; ++i) {
        if (ks * GROUPS + sgroup + i < KG) {
          next_s[i / 2] |= static_cast<uint32_t>(ps[i]) << (16 * (i & 1));
          if (p.zeros) next_z[i / 4] |= static_cast<uint32_t>(pz[i]) << (8 * (i & 3));
        }
      }
    }
  };
  auto put_scales = [&]() {
#pragma unroll
    for (int i = 0; i < PG; ++i) {
      // (keeps every use of the loads from moving up to them, a stage early)
      if (i % 2 == 0) asm volatile("" : "+r"(next_s[i / 2]));
      if (i % 4 == 0) asm volatile("" : "+r"(next_z[i / 4]));
      const uint32_t h = i % 2 ? next_s[i / 2] >> 16 : next_s[i / 2] & 0xffffu;
      const bool bf = BF || (XK != W4_F16 && p.out_bf16);
      const float sc = bf ? __uint_as_float(h << 16)
                          : __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
      const uint32_t z = p.zeros ? next_z[i / 4] >> (8 * (i % 4)) & 15u : 8u;
      table[i * WR] = make_float2(sc, __uint_as_float(zero_pair<BF>(z)));
    }
  };

  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // this lane's row of x in the products' columns; rows past the last read the
  // last one's values, in columns that are never stored
  const uint32_t x_row = sbase + lay.x + static_cast<uint32_t>(min(g, p.M - 1) * 64 + t * 16);

  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  if (segments > 0) load_scales(part_of(0, kw));
  for (int seg = 0; seg < segments; ++seg) {
    // ------------------------------------------------------- x of a segment
    const int first = ks0 + seg * p.segment;
    const int units = (min(ks1, first + p.segment) - first) * W4_UNITS;
    if (seg > 0) __syncthreads();  // every warp is done with the one before
    // 8 columns of a row of x a thread
    for (int i = threadIdx.x; i < units * 4 * p.M; i += blockDim.x) {
      const int m = i / (units * 4), c = i - m * (units * 4);
      const int k = first * W4_STAGE_K + c * 8;
      uint4 b = make_uint4(0, 0, 0, 0);
      if (k < p.K) {
        const uint8_t* src = static_cast<const uint8_t*>(p.x) +
                             (static_cast<int64_t>(m) * p.ldx + k) * XB;
        uint4 v;
        if constexpr (XB == 2) {
          v = *reinterpret_cast<const uint4*>(src);
        } else {
          const uint2 e = *reinterpret_cast<const uint2*>(src);
          v = make_uint4(e.x, e.y, 0, 0);
        }
        b = pair_x<XK>(v);
      }
      *reinterpret_cast<uint4*>(smem + lay.x + ((c >> 2) * p.M + m) * 64 + (c & 3) * 16) = b;
    }
    __syncthreads();
    // -------------------------------------------------------------- stages
    const int end = part_of(seg, kw + 1);
    for (int ks = part_of(seg, kw); ok && ks < end; ++ks) {
      put_scales();
      // (a segment's last stage loads its own scales again where the warp's
      // next part is not the next stage)
      const int after = ks + 1 < end ? ks + 1 : seg + 1 < segments ? part_of(seg + 1, kw) : ks;
      load_scales(after);
      __syncwarp();
      ok = __all_sync(0xffffffffu, wait_bounded_lazy(full0 + 8 * s, phase, ctl, WAIT_MMA_FULL));
      if (!ok) break;
      const uint32_t codes = ring + s * STAGE + g * 128;
      const uint32_t swz = static_cast<uint32_t>(g << 4 | t << 2);
      const uint32_t xu = static_cast<uint32_t>((ks - first) * W4_UNITS * p.M * 64);
      const uint32_t x_step = static_cast<uint32_t>(p.M * 64);
      const uint32_t tab = sbase + lay.table + (warp * (WR * GROUPS) + g) * 8;
      float part[4];                // a group's sums of products,
      float2 f[2];                  // its factors and zero points in rows g and g + 8
      uint32_t zh[2] = {0u, 0u};
      // (four units at a time: unrolled further, the loads all move to the
      // front and spill)
      constexpr int UB = 4;
#pragma unroll 1
      for (int u0 = 0; u0 < W4_UNITS; u0 += UB) {
#pragma unroll
        for (int ui = 0; ui < UB; ++ui) {
          const int u = u0 + ui;
          const bool start = ui % UPG == 0;  // of the group
          if (start) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f[h] = lds64f(tab + (u / UPG * WR + 8 * h) * 8);
              if constexpr (!BF) zh[h] = zero_pair_high(__float_as_uint(f[h].y));
            }
          }
          // rows 8 apart share their low three bits: the same swizzle
          const uint32_t off = codes + (swz ^ static_cast<uint32_t>(u << 4));
          uint32_t al[2], bl[2], ah[2], bh[2];
          spread_codes<BF>(p, lds32(off), __float_as_uint(f[0].y), zh[0], al, bl);
          spread_codes<BF>(p, lds32(off + 1024), __float_as_uint(f[1].y), zh[1], ah, bh);
          const uint32_t a[4] = {al[0], ah[0], al[1], ah[1]};
          const uint32_t b[4] = {bl[0], bh[0], bl[1], bh[1]};
          const uint4 x = lds128(x_row + xu + static_cast<uint32_t>(u) * x_step);
          mma_m16n8k16<BF>(part, a, x.x, x.y, start);
          mma_m16n8k16<BF>(part, b, x.z, x.w, false);
          if (ui % UPG == UPG - 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(f[i >> 1].x, part[i], acc[i]);
          }
        }
      }
      __syncwarp();
      issue_next(s);
      if (++s == S) {
        s = 0;
        phase ^= 1u;
      }
    }
  }
  grid_launch_dependents();
  if (!ok) {
    // a wait ran out: let every copy already issued land before the CTA exits
    for (int i = max(0, issued - S); i < issued; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(full0 + 8 * (i % S), static_cast<uint32_t>(i / S) & 1u) &&
             global_timer_ns() - t0 < ctl.timeout_ns) {
      }
    }
  }
  // Everything has been read: the partial sums take the rings' place.
  __syncthreads();
  const int pitch = w4_red_pitch(R);
  {
    float* red = reinterpret_cast<float*>(smem) + (kw * W4_X_ROWS + 2 * t) * pitch + WR * rw + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) red[(i & 1) * pitch + 8 * (i >> 1)] = acc[i];
  }
  __syncwarp();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each CTA of the cluster adds up its share of the rows of weights, over
  // the CTAs and parts of K in order.
  const int rows = R / p.splits;
  for (int i = threadIdx.x; i < rows * p.M; i += blockDim.x) {
    const int m = i / rows, r = rank * rows + i % rows;
    const uint32_t at0 = sbase + static_cast<uint32_t>((m * pitch + r) * 4);
    float v = 0.0f;
    for (int c = 0; c < p.splits; ++c) {
      const uint32_t from = p.splits > 1 ? map_to_cta(at0, static_cast<uint32_t>(c)) : at0;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const uint32_t addr = from + static_cast<uint32_t>(k * W4_X_ROWS * pitch * 4);
        float a;
        if (p.splits > 1)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a) : "r"(addr) : "memory");
        else
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(a) : "r"(addr) : "memory");
        v += a;
      }
    }
    if (p.x_scales) v *= p.x_scales[m];
    if (n0 + r < p.N) {
      if (p.out_bf16)
        store_out<OUT_BF16>(p.out, static_cast<int64_t>(m) * p.ldo + n0 + r, v);
      else
        store_out<OUT_F16>(p.out, static_cast<int64_t>(m) * p.ldo + n0 + r, v);
    }
  }
  __syncwarp();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// The variants of one kind of x (a translation unit each).
template <int XK>
const void* w4_kernel_of(int group) {
  return group == 32   ? reinterpret_cast<const void*>(&w4_gemm_kernel<XK, 32>)
         : group == 64 ? reinterpret_cast<const void*>(&w4_gemm_kernel<XK, 64>)
                       : reinterpret_cast<const void*>(&w4_gemm_kernel<XK, 128>);
}

}  // namespace sptg
