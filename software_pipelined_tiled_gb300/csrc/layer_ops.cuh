// layer_ops.cuh -- the C ABI of the operators around the dense products:
// residual addition with norm, products with 4-bit weights, products grouped
// by expert. Argument checks, kernel choice and launch; part of sptgemm.cu,
// whose device state, tensor maps and error texts it shares.
#pragma once

namespace {

struct TypeInfo {
  int bytes;
  const char* name;
  CUtensorMapDataType tma;
};

bool type_info(int type, TypeInfo& t) {
  switch (type) {
    case SPTG_T_F16: t = {2, "f16", CU_TENSOR_MAP_DATA_TYPE_FLOAT16}; return true;
    case SPTG_T_BF16: t = {2, "bf16", CU_TENSOR_MAP_DATA_TYPE_BFLOAT16}; return true;
    case SPTG_T_S8: t = {1, "s8", CU_TENSOR_MAP_DATA_TYPE_UINT8}; return true;
    case SPTG_T_E4M3: t = {1, "e4m3", CU_TENSOR_MAP_DATA_TYPE_UINT8}; return true;
    default: return false;
  }
}

int refuse(int status, const char* why) {
  t_last_error = why;
  return status;
}

bool multiple16(int64_t elements, int bytes) { return (elements * bytes) % 16 == 0; }

// A 3-D map: `inner` contiguous elements, rows `pitch` and planes `plane`
// bytes apart. Cached like the 2-D maps.
struct Map3dEntry {
  const void* base = nullptr;
  uint64_t dims[3] = {}, strides[2] = {};
  uint32_t box[3] = {};
  int dt = -1, swizzle = -1;
  CUtensorMap map;
};
constexpr int kMap3dCache = 32;
thread_local Map3dEntry t_maps3d[kMap3dCache];
thread_local int t_map3d_next = 0;

int make_map_3d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner,
                uint64_t rows, uint64_t planes, uint64_t pitch, uint64_t plane, uint32_t box_inner,
                uint32_t box_rows, uint32_t box_planes, CUtensorMapSwizzle swizzle) {
  for (const Map3dEntry& e : t_maps3d) {
    if (e.base == base && e.dims[0] == inner && e.dims[1] == rows && e.dims[2] == planes &&
        e.strides[0] == pitch && e.strides[1] == plane && e.box[0] == box_inner &&
        e.box[1] == box_rows && e.box[2] == box_planes && e.dt == static_cast<int>(dt) &&
        e.swizzle == static_cast<int>(swizzle)) {
      *map = e.map;
      return SPTG_OK;
    }
  }
  auto enc = tensor_map_encoder();
  if (!enc) return refuse(SPTG_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
  Map3dEntry n;
  n.base = base;
  n.dims[0] = inner;
  n.dims[1] = rows;
  n.dims[2] = planes;
  n.strides[0] = pitch;
  n.strides[1] = plane;
  n.box[0] = box_inner;
  n.box[1] = box_rows;
  n.box[2] = box_planes;
  n.dt = static_cast<int>(dt);
  n.swizzle = static_cast<int>(swizzle);
  const cuuint64_t dims[3] = {inner, rows, planes}, strides[2] = {pitch, plane};
  const cuuint32_t box[3] = {box_inner, box_rows, box_planes};
  const CUresult r = encode_tiled(enc, &n.map, dt, 3, base, dims, strides, box, swizzle);
  if (r != CUDA_SUCCESS) {
    char b[160];
    snprintf(b, sizeof(b), "cuTensorMapEncodeTiled failed (%d) for %llux%llux%llu", (int)r,
             (unsigned long long)planes, (unsigned long long)rows, (unsigned long long)inner);
    return refuse(SPTG_ERR_ARG, b);
  }
  *map = n.map;
  t_maps3d[t_map3d_next] = n;
  t_map3d_next = (t_map3d_next + 1) % kMap3dCache;
  return SPTG_OK;
}

// Launches with programmatic overlap (the kernels wait for the previous one
// before they touch memory), in clusters of `cluster` CTAs along x.
cudaError_t launch_op(const void* fn, dim3 grid, int threads, int smem, int cluster,
                      cudaStream_t stream, void** args) {
  cudaLaunchConfig_t lc;
  memset(&lc, 0, sizeof(lc));
  lc.gridDim = grid;
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  lc.attrs = attr;
  lc.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelExC(&lc, fn, args);
  ++t_launches;
  return e;
}

// No C++ exception leaves a C entry point (the tables and texts allocate).
template <typename F>
int guarded(F&& body) {
  try {
    t_launches = 0;
    return body();
  } catch (const std::bad_alloc&) {
    return SPTG_ERR_NOMEM;
  } catch (...) {
    return SPTG_ERR_LAUNCH;
  }
}

// Dimensions stop short of 2^31 by more than any tile, so that the kernels'
// 32-bit coordinates may run past an edge.
constexpr int64_t kMaxDim = (static_cast<int64_t>(1) << 31) - 4096;
constexpr const char* kDimText = "dimensions must be in [0, 2^31 - 4096]";

constexpr uint64_t kOpTimeoutNs = 2000ull * 1000000ull;

// Blocks of a kernel that an SM holds at once, and its registers a thread, by
// device, kernel, threads and shared memory.
struct Residency {
  int blocks, regs;
};
std::map<std::tuple<int, const void*, int, int>, Residency> g_residency;

int residency(Residency& out, int dev, const void* fn, int threads, int smem) {
  std::lock_guard<std::mutex> lk(g_mu);
  const auto key = std::make_tuple(dev, fn, threads, smem);
  const auto it = g_residency.find(key);
  if (it != g_residency.end()) {
    out = it->second;
    return SPTG_OK;
  }
  cudaFuncAttributes attr;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&out.blocks, fn, threads, smem);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, fn);
  if (e != cudaSuccess) return cuda_fail(e, "occupancy of a kernel");
  out.blocks = std::max(1, out.blocks);
  out.regs = attr.numRegs;
  g_residency[key] = out;
  return SPTG_OK;
}

// ------------------------------------------------------- residual and norm
int add_rms_norm(int64_t rows, int64_t cols, int in_type, int out_type, const void* x, int64_t ldx,
                 const void* r, int64_t ldr, const void* w, float eps, void* h, int64_t ldh,
                 void* y, int64_t ldy, float* scales, cudaStream_t stream, const sptg_config* cfg) {
  TypeInfo in, out;
  if ((in_type != SPTG_T_F16 && in_type != SPTG_T_BF16) || !type_info(in_type, in) ||
      !type_info(out_type, out) || (out.bytes == 2 && out_type != in_type))
    return refuse(SPTG_ERR_ARG, "rows are f16 or bf16, outputs s8, e4m3 or the rows' own type");
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return refuse(SPTG_ERR_ARG, kDimText);
  const int timeout_ms = cfg ? cfg->timeout_ms : 0, inject_stall = cfg ? cfg->inject_stall : 0;
  if (timeout_ms < 0 || (inject_stall != 0 && inject_stall != 1))
    return refuse(SPTG_ERR_ARG, "timeout_ms must not be negative, inject_stall 0 or 1");
  if (!(eps > 0.0f) || !(eps < INFINITY)) return refuse(SPTG_ERR_ARG, "eps must be positive and finite");
  if (rows == 0 || cols == 0) {
    set_config("kernel=none type=%s (empty output)", in.name, {});
    return SPTG_OK;
  }
  const bool quantised = out.bytes == 1;
  if (!x || !r || !w || !h || !y || (quantised && !scales)) return refuse(SPTG_ERR_ARG, "null pointer");
  if (ldx < cols || ldr < cols || ldh < cols || ldy < cols)
    return refuse(SPTG_ERR_ARG, "row pitches must be at least cols");
  const auto off = [](const void* p, unsigned bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
  };
  if (off(x, 2) || off(r, 2) || off(w, 2) || off(h, 2) || off(y, out.bytes) ||
      (quantised && off(scales, 4)))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  const int rc = device_info(di, dev);
  if (rc) return rc;
  const bool vectors = cols % 8 == 0 && ldx % 8 == 0 && ldr % 8 == 0 && ldh % 8 == 0 &&
                       ldy % 8 == 0 && !off(x, 16) && !off(r, 16) && !off(w, 16) && !off(h, 16) &&
                       !off(y, 8 * out.bytes);
  const int out_kind = out_type == SPTG_T_S8 ? NORM_S8 : out_type == SPTG_T_E4M3 ? NORM_E4M3 : NORM_16;
  // Rows up to 1024 elements: one to a warp. Wider ones: one to a block of as
  // many threads as it needs, or, where there are rows enough to go several
  // times through the GPU, rows through the ring kernel's blocks. Rows past
  // 16384 elements take the kernel for any width.
  const auto round32 = [](int64_t n) { return static_cast<int>((n + 31) / 32 * 32); };
  int kind = NORM_ANY, threads = 512, smem = 0, stages = 0, regs = 0;
  int64_t grid = rows;
  if (vectors && cols <= 1024) {
    kind = cols <= 512 ? NORM_WARP_2 : NORM_WARP_4;
    threads = 128;
    grid = (rows + 3) / 4;
  } else if (vectors && cols <= 16384) {
    // two groups of 8 elements a thread; four for rows of 2049 to 4096 elements
    // where there are rows to fill the GPU with (16384 rows of 4096: 71 us,
    // with two 75, through the ring 79)
    const bool four = cols > 2048 && cols <= 4096 && rows >= 4 * di.sm_count;
    kind = four ? NORM_BLOCK_4 : NORM_BLOCK_2;
    threads = four ? round32((cols / 8 + 3) / 4) : round32((cols / 8 + 1) / 2);
    // The ring kernel: three rows ahead, as many blocks as the GPU holds at once
    // (rows are dealt out to all blocks from the start; 16384 binary16 rows of 6144
    // to int8, two blocks to an SM by their registers: 117 us, with three 134 us).
    if (cols > 4096 && rows >= 3 * di.sm_count) {
      const int ring_threads = round32((cols / 8 + 3) / 4);
      const int ring_stages = 3;
      const int ring_smem = norm_ring_smem(static_cast<int>(cols), ring_stages);
      const void* ring = norm_variant(in_type == SPTG_T_BF16, out_kind, NORM_RING_4);
      Residency res;
      int rs = ensure_smem(dev, ring, norm_ring_smem(16384, 3));
      if (!rs) rs = residency(res, dev, ring, ring_threads, ring_smem);
      if (rs) return rs;
      const int64_t blocks = static_cast<int64_t>(res.blocks) * di.sm_count;
      if (rows >= 3 * blocks) {
        kind = NORM_RING_4;
        threads = ring_threads;
        stages = ring_stages;
        smem = ring_smem;
        grid = blocks;
        regs = res.regs;
      }
    }
  }
  const void* fn = norm_variant(in_type == SPTG_T_BF16, out_kind, kind);
  NormParams p{x, r, w, h, y, scales, ldx, ldr, ldh, ldy, rows, static_cast<int>(cols), eps,
               stages, di.error_word, timeout_ms ? timeout_ms * 1000000ull : kOpTimeoutNs, inject_stall};
  void* args[] = {&p};
  const cudaError_t e =
      launch_op(fn, dim3(static_cast<unsigned>(grid)), threads, smem, 1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "add_rms_norm launch");
  set_config("kernel=add_rms_norm type=%s out_bytes=%lld kind=%lld threads=%lld grid=%lld stages=%lld "
             "smem=%lld regs=%lld",
             in.name, {out.bytes, kind, threads, grid, stages, smem, regs});
  return SPTG_OK;
}

// ---------------------------------------------------------- 4-bit weights
// Rows of weights per CTA and CTAs sharing K (a cluster). For each cluster
// size the rows are cut so that the CTAs fill the GPU once to eight times, within
// `least` to `most`; the choice whose busiest SM has the least to do wins, in
// bytes of codes. The CTAs of the streaming kernel, two to an SM, share its rate:
// fewer and taller ones, one to an SM, do as well and start half as often (one row
// through 16384 x 4096: 148 of 112 rows 12.8 us, 256 of 64 rows 14.5 us), as long
// as an SM has twelve warps or so (128 of 64 rows, eight warps each, through
// 8192 x 8192: 19.1 us; 148 of 112 rows 13.6 us) and x need not be loaded in parts,
// between which a CTA waits (8 rows: 148 CTAs 15.7 us, 296 of half K 15.0 us).
// Clusters of 4 and 8 are placed two CTAs to an SM even where SMs are free (one row
// through 4096 x 4096: 148 CTAs of 112 rows 8.1 us, 256 of 64 rows 5.8 us). The tile
// kernel takes a stage in the same time whatever its rows. Starting a round of CTAs
// counts as 32 KB, a cluster's exchange as 16 KB.
struct W4Shape {
  int rows, splits;
};

W4Shape w4_shape(int64_t N, int64_t k_stages, bool tile, int64_t m_blocks, int64_t segment,
                 const int* slots) {
  constexpr int64_t step = 16, least = 64;
  const int64_t most = tile ? W4T_MAX_ROWS : W4_MAX_ROWS;
  const int per_sm = tile ? 1 : W4_CTAS_PER_SM;
  W4Shape best{static_cast<int>(most), 1};
  double best_t = 1e300;
  for (int i = 0; i < 4 && (1 << i) <= k_stages; ++i) {
    const int splits = 1 << i;
    for (int64_t fills = 1; fills <= 8; ++fills) {
      const int64_t room = slots[i] * fills / per_sm;
      const int64_t fit = (N * splits * m_blocks + room - 1) / room;
      const int64_t rows = std::min(most, std::max(least, (fit + step - 1) / step * step));
      const int64_t ctas = (N + rows - 1) / rows * splits * m_blocks;
      const int64_t rounds = (ctas + slots[i] - 1) / slots[i];
      // CTAs that the busiest SM gets, and warps at a time
      int64_t on_sm = (ctas * per_sm + slots[i] - 1) / slots[i];
      if (splits > 2) on_sm = rounds * per_sm;
      const int64_t warps = rows / W4_WARP_ROWS * W4_KW * std::min<int64_t>(on_sm, per_sm);
      const int64_t slice = (k_stages + splits - 1) / splits;
      double stage = (tile ? W4T_MAX_ROWS : rows) * 128.0;
      if (!tile && warps < 12) stage *= 12.0 / static_cast<double>(warps);
      if (!tile && on_sm == 1 && slice > segment) stage *= 1.25;
      const double t = static_cast<double>(on_sm * slice) * stage +
                       static_cast<double>(rounds) * (32768 + (splits > 1 ? 16384 : 0));
      if (t < best_t * 0.999) {
        best_t = t;
        best = {static_cast<int>(rows), splits};
      }
    }
  }
  return best;
}

// CTAs resident at once in clusters of 1, 2, 4 and 8, by device and kernel.
struct W4Slots {
  int n[4];
};
std::map<std::pair<int, const void*>, W4Slots> g_w4_slots;

W4Slots w4_slots(int dev, const void* fn, int per_sm, int threads, int sm_count) {
  std::lock_guard<std::mutex> lk(g_mu);
  const auto it = g_w4_slots.find({dev, fn});
  if (it != g_w4_slots.end()) return it->second;
  W4Slots w;
  w.n[0] = per_sm * sm_count;
  for (int i = 1; i < 4; ++i) {
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof(lc));
    lc.gridDim = dim3(static_cast<unsigned>(sm_count >> i << i), 1, 1);
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = 225 * 1024 / per_sm;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &lc) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = w.n[0] >> i;
    }
    w.n[i] = std::min(w.n[0], n << i);
  }
  g_w4_slots[{dev, fn}] = w;
  return w;
}

int gemm_w4(int64_t M, int64_t N, int64_t K, int group, int x_type, int out_type, const void* X,
            int64_t ldx, const float* x_scales, const uint8_t* codes, int64_t ldw,
            const void* scales, const uint8_t* zeros, void* Y, int64_t ldy, cudaStream_t stream) {
  TypeInfo xt, ot;
  if (!type_info(x_type, xt) || !type_info(out_type, ot) || ot.bytes != 2 ||
      (xt.bytes == 2 && x_type != out_type))
    return refuse(SPTG_ERR_ARG, "x is f16 or bf16 (and so is Y), or s8 or e4m3 (Y f16 or bf16)");
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return refuse(SPTG_ERR_ARG, kDimText);
  if (group != 32 && group != 64 && group != 128)
    return refuse(SPTG_ERR_ARG, "groups of 32, 64 or 128 columns");
  if (K % group != 0) return refuse(SPTG_ERR_ARG, "K must be a multiple of the group");
  if (M == 0 || N == 0) {
    set_config("kernel=none type=%s (empty output)", xt.name, {});
    return SPTG_OK;
  }
  if (!Y || (K > 0 && (!X || !codes || !scales))) return refuse(SPTG_ERR_ARG, "null pointer");
  if (xt.bytes == 1 && !x_scales) return refuse(SPTG_ERR_ARG, "8-bit rows need their scales");
  if (xt.bytes == 2 && x_scales) return refuse(SPTG_ERR_ARG, "16-bit rows take no scales");
  if (ldy < N || (K > 0 && (ldx < K || ldw < K / 2)) || ldx > INT32_MAX || ldw > INT32_MAX)
    return refuse(SPTG_ERR_ARG, "row pitches must satisfy ldx >= K, ldw >= K / 2, ldy >= N (< 2^31)");
  if ((reinterpret_cast<uintptr_t>(Y) & 1u) || (reinterpret_cast<uintptr_t>(scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(x_scales) & 3u))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  if (K > 0 && (!aligned16(X) || !aligned16(codes) || !multiple16(ldx, xt.bytes) || ldw % 16 != 0))
    return refuse(SPTG_ERR_ALIGN, "x and the codes need 16-byte aligned bases and row pitches");
  int dev = 0;
  DeviceInfo di;
  int rc = device_info(di, dev);
  if (rc) return rc;
  if (K == 0) {  // the empty sum
    const cudaError_t e = cudaMemset2DAsync(Y, static_cast<size_t>(ldy) * 2, 0,
                                            static_cast<size_t>(N) * 2, M, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset2DAsync");
    set_config("kernel=zero-fill type=%s", xt.name, {});
    return SPTG_OK;
  }
  // Up to 8 rows of x: the streaming kernel. More: the tensor-core tile kernel
  // with 16, 32 or 64 rows, in blocks of 64 (groups of 32 columns: of 32) that
  // each pass over the weights. Through 8192 x 8192 (bf16, groups of 128) the
  // streaming kernel takes 13.6 us for one row and 15.0 us for 8, the tile kernel
  // 15.8 us for 8 and 9 and 16.4 us for 16; through 4096 x 4096 5.8 and 7.0 us, the
  // tile kernel 7.7 us for 8 and 8.0 us for 16.
  const bool tile = M > 8;
  const int nt = M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : w4t_max_ntok(group);
  const int64_t m_blocks = (M + nt - 1) / nt;
  int xk;
  const void* fn;
  switch (x_type) {
    case SPTG_T_BF16:
      xk = W4_BF16;
      fn = tile ? w4_tile_kernel_bf16(nt, group) : w4_kernel_bf16(group);
      break;
    case SPTG_T_F16:
      xk = W4_F16;
      fn = tile ? w4_tile_kernel_f16(nt, group) : w4_kernel_f16(group);
      break;
    case SPTG_T_S8:
      xk = W4_S8;
      fn = tile ? w4_tile_kernel_s8(nt, group) : w4_kernel_s8(group);
      break;
    default:
      xk = W4_E4M3;
      fn = tile ? w4_tile_kernel_e4m3(nt, group) : w4_kernel_e4m3(group);
      break;
  }
  const int64_t k_stages = (K + W4_STAGE_K - 1) / W4_STAGE_K;
  rc = ensure_smem(dev, fn, 232448);  // the ring's size differs from call to call
  if (rc) return rc;
  const int threads = tile ? w4t_threads(xk, nt) : 32 * W4_MAX_WARPS;
  const W4Slots slots = w4_slots(dev, fn, tile ? 1 : W4_CTAS_PER_SM, threads, di.sm_count);
  // Stages of x that two fifths of a streaming CTA's shared memory hold.
  const int budget = (224 << 10) / W4_CTAS_PER_SM - 1024;
  const int live_m = static_cast<int>(std::min<int64_t>(M, W4_X_ROWS));
  const int x_stage = live_m * W4_STAGE_K * 2;
  const int x_stages = (budget * 2 / 5) / x_stage;
  const W4Shape shape = w4_shape(N, k_stages, tile, m_blocks, x_stages, slots.n);
  const int rows = shape.rows, splits = shape.splits;
  const int64_t n_tiles = (N + rows - 1) / rows;
  if (n_tiles * splits > INT32_MAX) return refuse(SPTG_ERR_ARG, "too many columns");
  W4Params p;
  int smem, launch_threads = threads;
  if (tile) {
    // as many stages of codes as fit beside three or four of x
    p.segment = w4t_x_stages(nt);
    p.stages = W4T_MAX_STAGES;
    while (p.stages > W4T_MIN_STAGES && w4t_smem(xk, nt, rows, p.stages, p.segment) > 232448) --p.stages;
    smem = w4t_smem(xk, nt, rows, p.stages, p.segment);
  } else {
    // Rings of at least two stages, a segment of x (a multiple of the parts
    // of K that warps take), the rings with what is left.
    const int kw = W4_KW;
    const int slice = static_cast<int>((k_stages + splits - 1) / splits);
    p.segment = std::max(kw, x_stages / kw * kw);
    p.segment = std::min(p.segment, (slice + kw - 1) / kw * kw);
    while (p.segment > kw && w4_layout(group, rows, 2, p.segment, live_m).total > budget)
      p.segment -= kw;
    p.stages = W4_MAX_STAGES;
    while (p.stages > 2 && w4_layout(group, rows, p.stages, p.segment, live_m).total > budget)
      --p.stages;
    const W4Layout lay = w4_layout(group, rows, p.stages, p.segment, live_m);
    smem = lay.total + 1024;
    launch_threads = 32 * lay.warps;
  }
  CUtensorMap mw, mx;
  rc = make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, codes, K / 2, N, W4_STAGE_K / 2,
                   tile ? rows : W4_WARP_ROWS, CU_TENSOR_MAP_SWIZZLE_128B, ldw);
  if (!rc && tile) {
    if (xt.bytes == 1)
      rc = make_map_2d(&mx, xt.tma, 1, X, K, M, W4_STAGE_K, nt, CU_TENSOR_MAP_SWIZZLE_NONE, ldx);
    else
      rc = make_map_2d(&mx, xt.tma, 2, X, K, M, 64, nt, CU_TENSOR_MAP_SWIZZLE_128B, ldx);
  }
  if (rc) return rc;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.x = X;
  p.ldx = ldx;
  p.rows = rows;
  p.splits = splits;
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = zeros;
  p.x_scales = x_scales;
  p.out = static_cast<uint16_t*>(Y);
  p.ldo = ldy;
  p.out_bf16 = out_type == SPTG_T_BF16;
  // a lane's groups are one load of up to 8 bytes of scales and 4 of zeros
  p.wide = K % W4_STAGE_K == 0 && aligned16(scales) && (reinterpret_cast<uintptr_t>(zeros) & 7u) == 0;
  p.mask_lo = 0x000f000fu;
  p.mask_hi = 0x00f000f0u;
  p.mask_tile = x_type == SPTG_T_BF16 ? p.mask_lo : 0x00f0000fu;
  p.magic = x_type == SPTG_T_BF16 ? 0x43004300u : 0x64006400u;
  p.error_word = di.error_word;
  p.timeout_ns = kOpTimeoutNs;
  void* tile_args[] = {&mw, &mx, &p};
  void* stream_args[] = {&mw, &p};
  // a grid is at most 65535 high: more rows take several launches
  for (int64_t first = 0; first < m_blocks; first += 65535) {
    p.m_first = static_cast<int>(first * nt);
    const unsigned high = static_cast<unsigned>(std::min<int64_t>(65535, m_blocks - first));
    const cudaError_t e = launch_op(fn, dim3(static_cast<unsigned>(n_tiles * splits), high),
                                    launch_threads, smem, splits, stream, tile ? tile_args : stream_args);
    if (e != cudaSuccess) return cuda_fail(e, "gemm_w4 launch");
  }
  set_config("kernel=w4 type=%s x_rows=%lld group=%lld rows=%lld splits=%lld stages=%lld grid=%lld "
             "m_blocks=%lld threads=%lld segment=%lld smem=%lld",
             xt.name, {nt, group, rows, splits, p.stages, n_tiles * splits, m_blocks, launch_threads,
                       p.segment, smem});
  return SPTG_OK;
}

// -------------------------------------------------------- grouped products
// One of the three grouped products. `a` is the features' operand (W, or dY
// for dW), `b` the ragged side's (X or dY; X for dW).
int grouped(int mode, int64_t E, int64_t T, int64_t N, int64_t K, int dtype, const int32_t* offsets,
            const void* a, int64_t lda, const void* b, int64_t ldb, void* out, int64_t ldo,
            cudaStream_t stream) {
  DtypeInfo d;
  if (!dtype_info(dtype, d) || d.is_int8) return refuse(SPTG_ERR_ARG, "grouped products take the float dtypes");
  if (E < 0 || T < 0 || N < 0 || K < 0 || T > kMaxDim || N > kMaxDim || K > kMaxDim)
    return refuse(SPTG_ERR_ARG, kDimText);
  if (E > GROUPED_MAX_EXPERTS) return refuse(SPTG_ERR_ARG, "at most 1024 experts");
  // columns of the output and length of the sum (dW: the rows)
  const int64_t cols = mode == GROUPED_Y ? N : K;
  const int64_t sum = mode == GROUPED_Y ? K : N;
  const bool dw = mode == GROUPED_DW;
  if (cols == 0 || (dw ? E == 0 || N == 0 : T == 0)) {
    set_config("kernel=none dtype=%s (empty output)", d.name, {});
    return SPTG_OK;
  }
  if (!out) return refuse(SPTG_ERR_ARG, "null pointer");
  const int64_t b_cols = dw ? K : sum;
  const bool nothing = dw ? T == 0 : (sum == 0 || E == 0);
  if (!nothing && (!a || !b || !offsets)) return refuse(SPTG_ERR_ARG, "null pointer");
  if (ldo < cols || ldo > INT32_MAX || (!nothing && (ldb < b_cols || ldb > INT32_MAX || (dw && (lda < N || lda > INT32_MAX)))))
    return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths (< 2^31)");
  if (!aligned16(out) || !multiple16(cols, d.out_bytes) || !multiple16(ldo, d.out_bytes) ||
      !multiple16(N, d.in_bytes) || !multiple16(K, d.in_bytes) ||
      (!nothing && (!aligned16(a) || !aligned16(b) || !multiple16(ldb, d.in_bytes) ||
                    (dw && !multiple16(lda, d.in_bytes)))))
    return refuse(SPTG_ERR_ALIGN, "TMA needs 16-byte aligned bases and row pitches");
  if (!nothing && (reinterpret_cast<uintptr_t>(offsets) & 3u))
    return refuse(SPTG_ERR_ALIGN, "offsets not aligned to their type");
  // Tiles up to 64 rows wide (and a deeper ring of weights) where the experts
  // have few rows on average, else up to 256. Products of 2048 x 2048 bf16 weights,
  // with 64 and 256: 8 experts of 16 rows on average 14.9 and 15.9 us, of 32 15.2
  // and 16.6 us, of 64 20.5 and 17.7 us; 64 experts of 16 rows 79.9 and 86.5 us,
  // of 32 87.1 and 88.3 us, of 64 95.1 and 91.5 us, of 128 139 and 102 us.
  const int tt = (!dw && T <= 32 * E) ? 64 : 256;
  const int64_t F = mode == GROUPED_DX ? K : N;
  const int64_t nf = (F + 255) / 256;
  const int64_t tiles = dw ? E * nf * ((K + 255) / 256) : nf * (T / tt + E + 2);
  if (tiles > INT32_MAX / 2) return refuse(SPTG_ERR_ARG, "too many tiles");
  int dev = 0;
  DeviceInfo di;
  int rc = device_info(di, dev);
  if (rc) return rc;
  if (nothing) {  // empty sums
    const int64_t rows = dw ? E * N : T;
    const cudaError_t e = cudaMemset2DAsync(out, static_cast<size_t>(ldo) * d.out_bytes, 0,
                                            static_cast<size_t>(cols) * d.out_bytes, rows, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset2DAsync");
    set_config("kernel=zero-fill dtype=%s", d.name, {});
    return SPTG_OK;
  }
  KernelVariant v;
  if (mode == GROUPED_Y)
    v = d.in_bf16 ? grouped_variant_y_bf16(d.out_kind, tt) : grouped_variant_y_f16(d.out_kind, tt);
  else if (mode == GROUPED_DX)
    v = d.in_bf16 ? grouped_variant_dx_bf16(d.out_kind, tt) : grouped_variant_dx_f16(d.out_kind, tt);
  else
    v = d.in_bf16 ? grouped_variant_dw_bf16(d.out_kind, tt) : grouped_variant_dw_f16(d.out_kind, tt);
  CUtensorMap ma, mb, mb4;
  if (dw) {
    rc = make_map_2d(&ma, d.in_tma, 2, a, N, T, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, lda);
    if (!rc) rc = make_map_2d(&mb, d.in_tma, 2, b, K, T, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, ldb);
    if (!rc)  // the output
      rc = make_map_3d(&mb4, d.out_tma, out, K, N, E, K * d.out_bytes, N * K * d.out_bytes,
                       128 / d.out_bytes, 32, 1, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    rc = make_map_3d(&ma, d.in_tma, a, K, N, E, K * 2, N * K * 2, 64, mode == GROUPED_Y ? 128 : 64, 1,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (!rc) rc = make_map_2d(&mb, d.in_tma, 2, b, sum, T, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, ldb);
    if (!rc) rc = make_map_2d(&mb4, d.in_tma, 2, b, sum, T, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B, ldb);
  }
  if (rc) return rc;
  rc = ensure_smem(dev, v.fn, v.smem);
  if (rc) return rc;
  GroupedParams p;
  p.experts = static_cast<int>(E);
  p.T = static_cast<int>(T);
  p.F = static_cast<int>(F);
  p.C = static_cast<int>(dw ? K : sum);
  p.offsets = offsets;
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.lda = lda;
  p.ldb = ldb;
  p.out = out;
  p.ldo = ldo;
  p.keep_weights = tt == 256;
  p.error_word = di.error_word;
  p.timeout_ns = kOpTimeoutNs;
  const int64_t pairs = std::min<int64_t>(tiles, pair_slots(dev, v, di.sm_count));
  void* args[] = {&ma, &mb, &mb4, &p};
  const cudaError_t e =
      launch_op(v.fn, dim3(static_cast<unsigned>(2 * pairs)), v.threads, v.smem, 2, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "grouped product launch");
  set_config("kernel=grouped dtype=%s mode=%lld experts=%lld tile_n=%lld stages=%lld grid=%lld smem=%lld",
             d.name, {mode, E, tt, v.stages, 2 * pairs, v.smem});
  return SPTG_OK;
}

}  // namespace

extern "C" {

int sptg_add_rms_norm(int64_t rows, int64_t cols, sptg_type in_type, sptg_type out_type,
                      const void* x, int64_t ldx, const void* residual, int64_t ldr,
                      const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                      float* scales, void* stream) {
  return sptg_add_rms_norm_ex(rows, cols, in_type, out_type, x, ldx, residual, ldr, weight, eps, h,
                              ldh, y, ldy, scales, stream, nullptr);
}

int sptg_add_rms_norm_ex(int64_t rows, int64_t cols, sptg_type in_type, sptg_type out_type,
                         const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                         float* scales, void* stream, const sptg_config* cfg) {
  return guarded([&] {
    return add_rms_norm(rows, cols, in_type, out_type, x, ldx, residual, ldr, weight, eps, h, ldh,
                        y, ldy, scales, static_cast<cudaStream_t>(stream), cfg);
  });
}

int sptg_gemm_w4(int64_t M, int64_t N, int64_t K, int group, sptg_type x_type, sptg_type out_type,
                 const void* X, int64_t ldx, const float* x_scales, const uint8_t* codes,
                 int64_t ldw, const void* scales, const uint8_t* zeros, void* Y, int64_t ldy,
                 void* stream) {
  return guarded([&] {
    return gemm_w4(M, N, K, group, x_type, out_type, X, ldx, x_scales, codes, ldw, scales, zeros, Y,
                   ldy, static_cast<cudaStream_t>(stream));
  });
}

int sptg_grouped_gemm(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                      const int32_t* offsets, const void* X, int64_t ldx, const void* W, void* Y,
                      int64_t ldy, void* stream) {
  return guarded([&] {
    return grouped(GROUPED_Y, E, T, N, K, dtype, offsets, W, 0, X, ldx, Y, ldy,
                   static_cast<cudaStream_t>(stream));
  });
}

int sptg_grouped_gemm_dx(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                         const int32_t* offsets, const void* dY, int64_t lddy, const void* W,
                         void* dX, int64_t lddx, void* stream) {
  return guarded([&] {
    return grouped(GROUPED_DX, E, T, N, K, dtype, offsets, W, 0, dY, lddy, dX, lddx,
                   static_cast<cudaStream_t>(stream));
  });
}

int sptg_grouped_gemm_dw(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                         const int32_t* offsets, const void* dY, int64_t lddy, const void* X,
                         int64_t ldx, void* dW, void* stream) {
  return guarded([&] {
    return grouped(GROUPED_DW, E, T, N, K, dtype, offsets, dY, lddy, X, ldx, dW, K,
                   static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
