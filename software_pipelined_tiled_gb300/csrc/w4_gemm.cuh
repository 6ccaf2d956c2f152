// w4_gemm.cuh -- products of a few rows with 4-bit weights and group scales.
//
//   Y[m, n] = xs[m] * sum_g s[n, g] * sum_{k in group g} x[m, k] * (w[n, k] - z[n, g])
//
// w: 4-bit codes 0 ... 15, two to a byte along K (the even column in the low
// half); s: a 16-bit scale for each row of weights and group of G = 32, 64 or
// 128 columns; z: a zero point 0 ... 15 for each group, or 8 everywhere; x: 16
// bits, or 8 bits (int8, e4m3) with a 32-bit scale xs for each row.
//
// Exactness: w - z is an integer of magnitude at most 15 and is formed exactly
// in the 16-bit type (a code under the exponent of 128 in bfloat16, of 1024 in
// binary16, less the zero point under the same exponent); 8-bit x is exact in
// binary16. The tensor core multiplies these and adds in 32 bits; a group's
// sum is scaled in 32 bits and added to the running sum in 32 bits. The only
// rounding to 16 bits is that of Y.
//
// Memory-bound for few rows: N * K / 2 bytes of codes, each read once. A CTA
// takes 128 rows of weights and a range of K; a producer warp streams ring
// stages of 256 columns (128 rows x 128 bytes of codes, 128-byte swizzled,
// and the same columns of the 8 * NT rows of x) with the tensor-copy engine;
// eight consumer warps each hold 16 rows of weights against all rows of x.
// The range of K may be split over the CTAs of a cluster, whose partial sums
// meet through distributed shared memory in CTA order (no atomics: the result
// does not depend on timing).
//
// The multiply is the warp-wide 16 x 8 x 16 instruction, whose operands live
// in registers: weights are widened in registers and never stored, and with 8
// rows of x the instruction's rate is far above what memory delivers (a
// tcgen05 instruction would need the widened weights in shared memory: four
// times the codes' bytes written and read there).
//
// Order within K: the products' sum does not depend on which columns share an
// instruction, as long as both operands agree. Lane (g, t) = (lane / 4, lane
// mod 4) of a warp reads one 32-bit word of codes -- columns 8t ... 8t + 7 of
// a unit of 32 columns -- for its rows g and g + 8. Masking the word with
// 0x000f000f after shifts by 0, 4, 8, 12 leaves the column pairs (0, 4),
// (1, 5), (2, 6), (3, 7), which feed two instructions; x's eight values are
// paired the same way.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sptg {

// Rows of x as they lie in memory. 16-bit x multiplies in its own type, 8-bit
// x in binary16.
enum W4X : int { W4_BF16 = 0, W4_F16 = 1, W4_S8 = 2, W4_E4M3 = 3 };

constexpr int W4_ROWS = 128;      // rows of weights per CTA
constexpr int W4_STAGE_K = 256;   // columns per ring stage
constexpr int W4_UNITS = 8;       // units of 32 columns in a stage
constexpr int W4_CONSUMERS = 8;   // warps of 16 rows of weights
constexpr int W4_THREADS = 32 * (W4_CONSUMERS + 1);
constexpr int W4_CODE_STAGE = W4_ROWS * W4_STAGE_K / 2;
constexpr int W4_MAX_STAGES = 8;
constexpr int W4_RED_PITCH = 132;  // 32-bit words between rows of x in the partial sums
constexpr int W4_BAR_BYTES = 2 * W4_MAX_STAGES * 8 + 16;

struct W4Params {
  int M, N, K;
  int stages;          // ring depth
  int splits;          // CTAs of the cluster, sharing K
  const uint16_t* scales;  // N x K / G
  const uint8_t* zeros;    // N x K / G, or null (8)
  const float* x_scales;   // M, or null (1)
  uint16_t* out;           // M rows of N, ldo apart
  int64_t ldo;
  int out_bf16;            // type of scales and out: bfloat16, else binary16
  unsigned int* error_word;
  uint64_t timeout_ns;
};

__host__ __device__ constexpr int w4_x_bytes(int xk) { return xk >= W4_S8 ? 1 : 2; }
__host__ __device__ constexpr int w4_x_stage(int xk, int nt) {
  return W4_STAGE_K * 8 * nt * w4_x_bytes(xk);
}
__host__ __device__ constexpr int w4_stage_bytes(int xk, int nt) {
  return W4_CODE_STAGE + w4_x_stage(xk, nt);
}
__host__ __device__ constexpr int w4_red_bytes(int nt) { return 8 * nt * W4_RED_PITCH * 4; }
__host__ __device__ constexpr int w4_smem(int xk, int nt, int stages) {
  const int ring = stages * w4_stage_bytes(xk, nt);
  const int red = w4_red_bytes(nt);
  return (ring > red ? ring : red) + W4_BAR_BYTES + 1024;
}

template <bool BF>
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  if constexpr (BF) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
  } else {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
}

// The eight codes of a word, less the zero point (given as the pair of
// magic | z), as the four column pairs (0,4), (1,5), (2,6), (3,7).
template <bool BF>
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t zz, uint32_t (&out)[4]) {
  constexpr uint32_t MAGIC = BF ? 0x43004300u : 0x64006400u;
#pragma unroll
  for (int p = 0; p < 4; ++p) out[p] = sub2<BF>(((w >> (4 * p)) & 0x000f000fu) | MAGIC, zz);
}

// This lane's eight values of x of one unit, in the same column pairs.
template <int XK>
__device__ __forceinline__ void load_x(uint32_t addr, uint32_t (&b)[4]) {
  if constexpr (XK == W4_BF16 || XK == W4_F16) {
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
    b[0] = __byte_perm(v[0], v[2], 0x5410);
    b[1] = __byte_perm(v[0], v[2], 0x7632);
    b[2] = __byte_perm(v[1], v[3], 0x5410);
    b[3] = __byte_perm(v[1], v[3], 0x7632);
  } else {
    uint32_t v0, v1;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v0), "=r"(v1) : "r"(addr));
    const uint32_t lo = __byte_perm(v0, v1, 0x5140);  // bytes 0, 4, 1, 5
    const uint32_t hi = __byte_perm(v0, v1, 0x7362);  // bytes 2, 6, 3, 7
    if constexpr (XK == W4_S8) {
      // a byte with its sign bit flipped is b + 128; under the exponent byte
      // 0x64 it is 1024 + b + 128 in binary16, and 1152 less leaves b
      constexpr uint32_t E = 0x64646464u, BIAS = 0x64806480u;
      const uint32_t l = lo ^ 0x80808080u, h = hi ^ 0x80808080u;
      b[0] = sub2<false>(__byte_perm(l, E, 0x4140), BIAS);
      b[1] = sub2<false>(__byte_perm(l, E, 0x4342), BIAS);
      b[2] = sub2<false>(__byte_perm(h, E, 0x4140), BIAS);
      b[3] = sub2<false>(__byte_perm(h, E, 0x4342), BIAS);
    } else {
      const uint32_t q[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw r =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q[i]), __NV_E4M3);
        b[i] = static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
      }
    }
  }
}

template <int XK, int NT, int G>
__global__ void __launch_bounds__(W4_THREADS)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const W4Params p) {
  constexpr bool BF = XK == W4_BF16;
  constexpr int XB = w4_x_bytes(XK);
  constexpr int GROUPS = W4_STAGE_K / G;      // groups in a stage
  constexpr int UPG = G / 32;                 // units in a group
  constexpr int SREGS = 2 * GROUPS / 4;       // scale words per lane and stage
  constexpr int STAGE = w4_stage_bytes(XK, NT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = p.stages;
  const uint32_t sbase = smem_addr(smem);
  const int ring = S * STAGE > w4_red_bytes(NT) ? S * STAGE : w4_red_bytes(NT);
  const uint32_t bar0 = sbase + ring;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (W4_MAX_STAGES + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + ring + 2 * W4_MAX_STAGES * 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % p.splits;  // = the CTA's rank in its cluster
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * W4_ROWS;
  const int m0 = static_cast<int>(blockIdx.y) * 8 * NT;
  // this CTA's stages of K
  const int KS = (p.K + W4_STAGE_K - 1) / W4_STAGE_K;
  const int ks0 = static_cast<int>(static_cast<int64_t>(KS) * rank / p.splits);
  const int ks1 = static_cast<int>(static_cast<int64_t>(KS) * (rank + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), W4_CONSUMERS);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensor_map(&tmW);
    prefetch_tensor_map(&tmX);
  }
  __syncthreads();
  // warm L2 with the first stages of codes while the previous kernel drains
  // (the loads proper wait for it)
  if (threadIdx.x == 32 * W4_CONSUMERS && m0 == 0)
    for (int ks = ks0; ks < min(ks1, ks0 + S); ++ks) tma_prefetch_l2_2d(&tmW, ks * (W4_STAGE_K / 2), n0);
  grid_dependency_wait();
  const WaitCtl ctl{p.timeout_ns, p.error_word, abort_flag};
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;

  if (warp == W4_CONSUMERS) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one_sync();
    // codes are read once unless several blocks of rows of x pass over them
    const uint64_t pol_w = gridDim.y > 1 ? policy_evict_last() : policy_evict_first();
    const uint64_t pol_x = policy_evict_last();
    int issued = 0;
    bool ok = true;
    int s = 0;
    uint32_t round = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
      if (round > 0 && !__all_sync(0xffffffffu, wait_bounded(empty_bar(s), (round & 1u) ^ 1u, ctl,
                                                              WAIT_PRODUCER_EMPTY))) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(full_bar(s), STAGE);
        tma_load_2d(sbase + s * STAGE, &tmW, full_bar(s), ks * (W4_STAGE_K / 2), n0, pol_w);
        tma_load_3d(sbase + s * STAGE + W4_CODE_STAGE, &tmX, full_bar(s), 0, m0, ks * W4_UNITS,
                    pol_x);
      }
      ++issued;
      if (++s == S) {
        s = 0;
        ++round;
      }
    }
    grid_launch_dependents();
    if (!ok) {
      // let every copy already issued land before the CTA can exit
      for (int i = max(0, issued - S); i < issued; ++i) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(full_bar(i % S), static_cast<uint32_t>(i / S) & 1u) &&
               global_timer_ns() - t0 < ctl.timeout_ns) {
        }
      }
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int row = n0 + 16 * warp + g;  // and row + 8
    const int64_t KG = p.K / G;
    // Lane t of a quad loads the scales (and zero points) j = t, t + 4, ... of
    // the stage's 2 * GROUPS: j < GROUPS are row g's, the others row g + 8's.
    auto load_scales = [&](int ks, uint32_t (&sv)[SREGS]) {
#pragma unroll
      for (int i = 0; i < SREGS; ++i) {
        const int j = 4 * i + t;
        const int r = row + (j >= GROUPS ? 8 : 0);
        const int64_t gi = static_cast<int64_t>(ks) * GROUPS + (j % GROUPS);
        uint32_t v = 8u << 16;
        if (r < p.N && gi < KG) {
          const int64_t at = static_cast<int64_t>(r) * KG + gi;
          const uint32_t z = p.zeros ? (p.zeros[at] & 15u) : 8u;
          v = p.scales[at] | (z << 16);
        }
        sv[i] = v;
      }
    };
    uint32_t sv[SREGS];
    if (ks0 < ks1) load_scales(ks0, sv);
    int s = 0;
    uint32_t phase = 0;
    for (int ks = ks0; ks < ks1; ++ks) {
      uint32_t nv[SREGS];
      if (ks + 1 < ks1) load_scales(ks + 1, nv);
      if (!__all_sync(0xffffffffu, wait_bounded(full_bar(s), phase, ctl, WAIT_MMA_FULL))) break;
      const uint32_t codes = sbase + s * STAGE + (16 * warp + g) * 128 + 4 * t;
      const uint32_t xs = sbase + s * STAGE + W4_CODE_STAGE + lane * (8 * XB);
      float part[NT][4];
      uint32_t zlo = 0, zhi = 0;
      float slo = 0.0f, shi = 0.0f;
#pragma unroll
      for (int u = 0; u < W4_UNITS; ++u) {
        if (u % UPG == 0) {
          constexpr uint32_t MAGIC = BF ? 0x4300u : 0x6400u;
          const int jl = u / UPG, jh = GROUPS + u / UPG;
          const uint32_t vl = __shfl_sync(0xffffffffu, sv[jl / 4], (lane & 28) | (jl & 3));
          const uint32_t vh = __shfl_sync(0xffffffffu, sv[jh / 4], (lane & 28) | (jh & 3));
          zlo = (MAGIC | (vl >> 16)) * 0x00010001u;
          zhi = (MAGIC | (vh >> 16)) * 0x00010001u;
          const bool bf = BF || (XK != W4_F16 && p.out_bf16);
          slo = bf ? __uint_as_float(vl << 16) : __half2float(__ushort_as_half(vl & 0xffffu));
          shi = bf ? __uint_as_float(vh << 16) : __half2float(__ushort_as_half(vh & 0xffffu));
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[j][i] = 0.0f;
        }
        // rows g and g + 8 share their low three bits: the same swizzle
        const uint32_t off = static_cast<uint32_t>((u ^ g) << 4);
        uint32_t wl, wh;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wl) : "r"(codes + off));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wh) : "r"(codes + 8 * 128 + off));
        uint32_t al[4], ah[4];
        widen_codes<BF>(wl, zlo, al);
        widen_codes<BF>(wh, zhi, ah);
        const uint32_t a0[4] = {al[0], ah[0], al[1], ah[1]};
        const uint32_t a1[4] = {al[2], ah[2], al[3], ah[3]};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b[4];
          load_x<XK>(xs + (u * NT + j) * (256 * XB), b);
          mma_m16n8k16<BF>(part[j], a0, b[0], b[1]);
          mma_m16n8k16<BF>(part[j], a1, b[2], b[3]);
        }
        if (u % UPG == UPG - 1) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[j][0] += slo * part[j][0];
            acc[j][1] += slo * part[j][1];
            acc[j][2] += shi * part[j][2];
            acc[j][3] += shi * part[j][3];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
#pragma unroll
      for (int i = 0; i < SREGS; ++i) sv[i] = nv[i];
      if (++s == S) {
        s = 0;
        phase ^= 1u;
      }
    }
    // Every stage has been read: the ring becomes the buffer of partial sums.
    named_barrier_sync(1, 32 * W4_CONSUMERS);
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* r0 = red + (8 * j + 2 * t) * W4_RED_PITCH + 16 * warp + g;
      r0[0] = acc[j][0];
      r0[W4_RED_PITCH] = acc[j][1];
      r0[8] = acc[j][2];
      r0[W4_RED_PITCH + 8] = acc[j][3];
    }
  }
  __syncwarp();
  if (p.splits > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each CTA of the cluster adds up its share of the rows of weights, over
  // the CTAs in order.
  const int rows = W4_ROWS / p.splits;
  const int live_m = min(8 * NT, p.M - m0);
  for (int i = threadIdx.x; i < rows * live_m; i += W4_THREADS) {
    const int m = i / rows, r = rank * rows + i % rows;
    const uint32_t at = sbase + static_cast<uint32_t>((m * W4_RED_PITCH + r) * 4);
    float v = 0.0f;
    for (int c = 0; c < p.splits; ++c) {
      float a;
      if (p.splits > 1)
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(a)
                     : "r"(map_to_cta(at, static_cast<uint32_t>(c))));
      else
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(a) : "r"(at));
      v += a;
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

// The variants of one kind of x (a translation unit each).
template <int XK>
const void* w4_kernel_of(int nt, int group) {
#define SPTG_W4_CASE(NT_, G_) \
  if (nt == NT_ && group == G_) return reinterpret_cast<const void*>(&w4_gemm_kernel<XK, NT_, G_>)
  SPTG_W4_CASE(1, 32);
  SPTG_W4_CASE(1, 64);
  SPTG_W4_CASE(1, 128);
  SPTG_W4_CASE(2, 32);
  SPTG_W4_CASE(2, 64);
  SPTG_W4_CASE(2, 128);
  SPTG_W4_CASE(4, 32);
  SPTG_W4_CASE(4, 64);
  SPTG_W4_CASE(4, 128);
  SPTG_W4_CASE(8, 32);
  SPTG_W4_CASE(8, 64);
  SPTG_W4_CASE(8, 128);
#undef SPTG_W4_CASE
  return nullptr;
}

}  // namespace sptg
