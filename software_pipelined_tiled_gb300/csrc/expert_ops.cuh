// expert_ops.cuh -- the C ABI of the operators around an expert layer: routing,
// dispatch and combination of rows, and the gated residual with its norms.
// Argument checks, kernel choice and launch; part of sptgemm.cu, after
// layer_ops.cuh, whose helpers it shares.
#pragma once

namespace {

bool off_by(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Rows of these operators stop where a block's next piece is a 32-bit number still.
constexpr int64_t kMaxCols = static_cast<int64_t>(1) << 30;
constexpr const char* kRowText = "rows must be in [0, 2^31 - 4096], their elements in [0, 2^30]";

// 16-bit row types and their names.
bool row_type(int type, bool& bf16, const char*& name) {
  TypeInfo t;
  if (!type_info(type, t) || t.bytes != 2) return false;
  bf16 = type == SPTG_T_BF16;
  name = t.name;
  return true;
}

// Whether rows can be read in 16-byte pieces.
bool in_pieces(const void* p, int64_t ld) { return p == nullptr || (!off_by(p, 16) && ld % 8 == 0); }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ routing
bool route_type(int type, int& kind, int& bytes, const char*& name) {
  switch (type) {
    case SPTG_T_F16: kind = ROUTE_F16; bytes = 2; name = "f16"; return true;
    case SPTG_T_BF16: kind = ROUTE_BF16; bytes = 2; name = "bf16"; return true;
    case SPTG_T_F32: kind = ROUTE_F32; bytes = 4; name = "f32"; return true;
    default: return false;
  }
}

int route_sizes(int64_t rows, int64_t E, int top, float scale) {
  if (rows < 0 || rows > kMaxDim || E < 0) return refuse(SPTG_ERR_ARG, kDimText);
  if (E > ROUTE_MAX_EXPERTS) return refuse(SPTG_ERR_ARG, "at most 1024 experts");
  if (top < 1 || top > ROUTE_MAX_TOP || top > E || rows * top > kMaxDim)
    return refuse(SPTG_ERR_ARG, "top must be in [1, 16], no more than the experts, and rows * top below 2^31");
  if (!(scale > -INFINITY && scale < INFINITY)) return refuse(SPTG_ERR_ARG, "scale must be finite");
  return SPTG_OK;
}

int route_experts(int64_t rows, int64_t E, int top, int type, const void* logits, int64_t ld,
                  const float* bias, int sigmoid, int groups, int top_groups, int group_best,
                  int renorm, float scale, float* weights, int32_t* experts, cudaStream_t stream) {
  int kind, bytes;
  const char* name;
  if (!route_type(type, kind, bytes, name)) return refuse(SPTG_ERR_ARG, "logits are f16, bf16 or f32");
  int rc = route_sizes(rows, E, top, scale);
  if (rc) return rc;
  if (groups < 1 || groups > ROUTE_MAX_GROUPS || E % groups != 0)
    return refuse(SPTG_ERR_ARG, "groups must be in [1, 32] and divide the experts");
  if (top_groups < 1 || top_groups > groups || top > E / groups * top_groups)
    return refuse(SPTG_ERR_ARG, "top_groups must be in [1, groups] and its groups hold top experts");
  if (group_best != 1 && group_best != 2) return refuse(SPTG_ERR_ARG, "group_best must be 1 or 2");
  if ((sigmoid != 0 && sigmoid != 1) || (renorm != 0 && renorm != 1))
    return refuse(SPTG_ERR_ARG, "sigmoid and renormalize must be 0 or 1");
  if (rows == 0) {
    set_config("kernel=none type=%s (empty output)", name, {});
    return SPTG_OK;
  }
  if (!logits || !weights || !experts) return refuse(SPTG_ERR_ARG, "null pointer");
  if (ld < E) return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(logits, bytes) || off_by(bias, 4) || off_by(weights, 4) || off_by(experts, 4))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  // The fewest lanes a row (so the most rows a warp) that hold its experts, each
  // group's in lanes of its own, and a pick each. (More than 32 experts a lane: groups
  // whose number is no power of two, so that lanes stay empty.)
  RouteParams p;
  p.size = static_cast<int>(E) / groups;
  int group_slots = 1;
  while (group_slots < groups) group_slots *= 2;
  // (32768 rows of 128 bf16 logits: 12.7 us with 16 experts a lane, 15.1 us with 8; of 256: 22.8
  // us either way, one row 3.7 us with 8, 4.3 us with 16.)
  constexpr int lanes_of[] = {8, 8, 16, 32, 32, 32, 32}, per_of[] = {8, 16, 8, 8, 16, 32, 64};
  int v = 0;
  for (; v < 6; ++v)
    if (top <= lanes_of[v] && group_slots <= lanes_of[v] &&
        ceil_div(p.size, lanes_of[v] / group_slots) <= per_of[v])
      break;
  const int group_lanes = lanes_of[v] / group_slots, piece = 16 / bytes;
  p.lanes_log2 = 0;
  while ((1 << p.lanes_log2) < group_lanes) ++p.lanes_log2;
  // (whole 16-byte pieces to a lane)
  p.chunk = static_cast<int>(std::min<int64_t>(
      per_of[v], ceil_div(ceil_div(p.size, group_lanes), piece) * piece));
  p.wide = p.size % piece == 0 && p.chunk % piece == 0 && !off_by(logits, 16) && ld % piece == 0;
  p.wide_bias = p.size % 4 == 0 && p.chunk % 4 == 0 && !off_by(bias, 16);
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.bias = bias;
  p.weights = weights;
  p.experts = experts;
  p.E = static_cast<int>(E);
  p.top = top;
  p.sigmoid = sigmoid;
  p.renorm = renorm;
  p.scale = scale;
  p.groups = groups;
  p.top_groups = top_groups;
  p.group_best = group_best;
  // Several turns a warp fill its lanes with picks (32768 rows of 256 experts in
  // warps of one row each took 1.5 times as many instructions), where there
  // are rows for eight warps an SM all the same.
  p.slots_log2 = top <= 8 ? 3 : 4;
  const int at_once = 32 / lanes_of[v];
  const int64_t busy = rows / (static_cast<int64_t>(at_once) * 8 * di.sm_count);
  p.turns = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(lanes_of[v] >> p.slots_log2, busy)));
  const int64_t grid = ceil_div(rows, ROUTE_WARPS * at_once * p.turns);
  void* args[] = {&p};
  const cudaError_t e = launch_op(route_variant(kind, v), dim3(static_cast<unsigned>(grid)),
                                  32 * ROUTE_WARPS, 0, 1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "route_experts launch");
  set_config("kernel=route type=%s lanes=%lld per=%lld chunk=%lld wide=%lld turns=%lld grid=%lld", name,
             {lanes_of[v], per_of[v], p.chunk, p.wide, p.turns, grid});
  return SPTG_OK;
}

int route_dlogits(int64_t rows, int64_t E, int top, int type, const void* logits, int64_t ld,
                  const int32_t* experts, const float* dweights, int sigmoid, int renorm, float scale,
                  void* dlogits, int64_t ldd, cudaStream_t stream) {
  int kind, bytes;
  const char* name;
  if (!route_type(type, kind, bytes, name)) return refuse(SPTG_ERR_ARG, "logits are f16, bf16 or f32");
  int rc = route_sizes(rows, E, top, scale);
  if (rc) return rc;
  if ((sigmoid != 0 && sigmoid != 1) || (renorm != 0 && renorm != 1))
    return refuse(SPTG_ERR_ARG, "sigmoid and renormalize must be 0 or 1");
  if (rows == 0) {
    set_config("kernel=none type=%s (empty output)", name, {});
    return SPTG_OK;
  }
  if (!logits || !experts || !dweights || !dlogits) return refuse(SPTG_ERR_ARG, "null pointer");
  if (ld < E || ldd < E) return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(logits, bytes) || off_by(dlogits, bytes) || off_by(dweights, 4) || off_by(experts, 4))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  const int piece = 16 / bytes;
  RouteGradParams p{logits, ld, rows, experts, dweights, dlogits, ldd, static_cast<int>(E), top, sigmoid, renorm, scale, 0};
  p.wide = E % piece == 0 && ld % piece == 0 && ldd % piece == 0 && !off_by(logits, 16) && !off_by(dlogits, 16);
  const int slots = top <= 8 ? 8 : 16;
  const int64_t grid = ceil_div(rows, ROUTE_WARPS * 32 / slots);
  void* args[] = {&p};
  const cudaError_t e = launch_op(route_dlogits_variant(kind, slots), dim3(static_cast<unsigned>(grid)),
                                  32 * ROUTE_WARPS, 0, 1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "route_experts_dlogits launch");
  set_config("kernel=route_dlogits type=%s wide=%lld grid=%lld", name, {p.wide, grid});
  return SPTG_OK;
}

// ------------------------------------------------- rows to experts and back
int rows_sizes(int64_t rows, int64_t cols, int top) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxCols) return refuse(SPTG_ERR_ARG, kRowText);
  if (top < 1 || rows * top > kMaxDim) return refuse(SPTG_ERR_ARG, "top must be at least 1 and rows * top below 2^31");
  return SPTG_OK;
}

// Blocks that share a row's columns, so that few rows reach all SMs: about two an SM
// (4 rows of 2048 from 8 places each: 2.3 us).
unsigned column_parts(int64_t rows, int64_t pieces, int sm_count) {
  const int64_t most = ceil_div(pieces, ROWS_THREADS), want = ceil_div(2 * sm_count, rows);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>({most, want, 65535})));
}

// CTAs of a sort: a cluster of 16 where the GPU places one, else the 8 that it always does.
std::map<int, int> g_sort_cluster;

int sort_cluster(int dev, int& ctas) {
  const void* fn = dispatch_sort_variant();
  const int smem = sort_smem(DISPATCH_MAX_EXPERTS);
  int rc = ensure_smem(dev, fn, smem);
  if (rc) return rc;
  std::lock_guard<std::mutex> lk(g_mu);
  const auto it = g_sort_cluster.find(dev);
  if (it != g_sort_cluster.end()) {
    ctas = it->second;
    return SPTG_OK;
  }
  ctas = 8;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t lc;
    memset(&lc, 0, sizeof(lc));
    lc.gridDim = dim3(16, 1, 1);
    lc.blockDim = dim3(32 * SORT_WARPS, 1, 1);
    lc.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &lc) == cudaSuccess && n > 0) ctas = 16;
  }
  cudaGetLastError();
  g_sort_cluster[dev] = ctas;
  return SPTG_OK;
}

int dispatch_rows(int64_t rows, int64_t cols, int top, int64_t E, int type, const void* x, int64_t ldx,
                  const int32_t* experts, void* sorted, int64_t lds, int32_t* places, int32_t* offsets,
                  cudaStream_t stream) {
  bool bf16;
  const char* name;
  if (!row_type(type, bf16, name)) return refuse(SPTG_ERR_ARG, "rows are f16 or bf16");
  int rc = rows_sizes(rows, cols, top);
  if (rc) return rc;
  if (E < 0 || E > DISPATCH_MAX_EXPERTS) return refuse(SPTG_ERR_ARG, "at most 1024 experts");
  if (!offsets) return refuse(SPTG_ERR_ARG, "null pointer");
  const bool copies = rows > 0 && cols > 0;
  if (rows > 0 && (!experts || !places || (cols > 0 && (!x || !sorted))))
    return refuse(SPTG_ERR_ARG, "null pointer");
  if (copies && (ldx < cols || lds < cols))
    return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(x, 2) || off_by(sorted, 2) || off_by(experts, 4) || off_by(places, 4) || off_by(offsets, 4))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  if (rows == 0) {
    const cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    set_config("kernel=zero-fill type=%s", name, {});
    return SPTG_OK;
  }
  SortParams s;
  s.experts = experts;
  s.places = places;
  s.offsets = offsets;
  s.entries = rows * top;
  s.E = static_cast<int>(E);
  const bool aligned = cols % 8 == 0 && in_pieces(x, ldx) && in_pieces(sorted, lds);
  RowsParams p{};
  p.x = x;
  p.ldx = ldx;
  p.places = places;
  p.out = sorted;
  p.ldo = lds;
  p.out_rows = s.entries;
  p.cols = static_cast<int>(cols);
  p.top = top;
  const unsigned parts = column_parts(rows, ceil_div(cols + (aligned ? 0 : 7), 8), di.sm_count);
  void* args[] = {&p, &s};
  cudaError_t e;
  if (s.entries <= SMALL_ENTRIES) {
    e = launch_op(dispatch_small_variant(aligned), dim3(static_cast<unsigned>(rows + 1), parts), ROWS_THREADS, 0,
                  1, stream, args);
    if (e != cudaSuccess) return cuda_fail(e, "dispatch_rows launch");
    set_config("kernel=dispatch_small type=%s aligned=%lld parts=%lld", name, {aligned, parts});
    return SPTG_OK;
  }
  s.bits = 0;
  while (E >> s.bits) ++s.bits;
  int ctas = 0;
  rc = sort_cluster(dev, ctas);
  if (rc) return rc;
  s.per_warp = ceil_div(ceil_div(s.entries, ctas * SORT_WARPS), 32) * 32;
  void* sort_args[] = {&s};
  e = launch_op(dispatch_sort_variant(), dim3(static_cast<unsigned>(ctas)), 32 * SORT_WARPS, sort_smem(s.E), ctas,
                stream, sort_args);
  if (e != cudaSuccess) return cuda_fail(e, "dispatch_rows sort launch");
  if (copies) {
    e = launch_op(dispatch_copy_variant(aligned), dim3(static_cast<unsigned>(rows), parts), ROWS_THREADS, 0, 1,
                  stream, args);
    if (e != cudaSuccess) return cuda_fail(e, "dispatch_rows copy launch");
  }
  set_config("kernel=dispatch type=%s sort_ctas=%lld per_warp=%lld aligned=%lld", name,
             {ctas, s.per_warp, aligned});
  return SPTG_OK;
}

int combine_rows(int64_t rows, int64_t cols, int top, int64_t y_rows, int type, const void* y, int64_t ldy,
                 const int32_t* places, const float* weights, const void* base, int64_t ldb, void* out,
                 int64_t ldo, cudaStream_t stream) {
  bool bf16;
  const char* name;
  if (!row_type(type, bf16, name)) return refuse(SPTG_ERR_ARG, "rows are f16 or bf16");
  int rc = rows_sizes(rows, cols, top);
  if (rc) return rc;
  if (y_rows < 0 || y_rows > kMaxDim) return refuse(SPTG_ERR_ARG, kDimText);
  if (rows == 0 || cols == 0) {
    set_config("kernel=none type=%s (empty output)", name, {});
    return SPTG_OK;
  }
  if ((!y && y_rows > 0) || !places || !out) return refuse(SPTG_ERR_ARG, "null pointer");
  if ((y_rows > 0 && ldy < cols) || ldo < cols || (base && ldb < cols))
    return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(y, 2) || off_by(out, 2) || off_by(base, 2) || off_by(places, 4) || off_by(weights, 4))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  const bool aligned = cols % 8 == 0 && in_pieces(y, ldy) && in_pieces(out, ldo) && in_pieces(base, ldb);
  RowsParams p{};
  p.x = y;
  p.ldx = ldy;
  p.x_rows = y_rows;
  p.places = places;
  p.weights = weights;
  p.base = base;
  p.ldb = ldb;
  p.out = out;
  p.ldo = ldo;
  p.cols = static_cast<int>(cols);
  p.top = top;
  const unsigned parts = column_parts(rows, ceil_div(cols + (aligned ? 0 : 7), 8), di.sm_count);
  void* args[] = {&p};
  const cudaError_t e = launch_op(combine_rows_variant(bf16, aligned), dim3(static_cast<unsigned>(rows), parts),
                                  ROWS_THREADS, 0, 1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "combine_rows launch");
  set_config("kernel=combine type=%s aligned=%lld parts=%lld", name, {aligned, parts});
  return SPTG_OK;
}

int combine_rows_grad(int64_t rows, int64_t cols, int top, int64_t y_rows, int type, const void* dout,
                      int64_t ldd, const void* y, int64_t ldy, const int32_t* places, const float* weights,
                      void* dy, int64_t lddy, float* dweights, int zero_unnamed, cudaStream_t stream) {
  bool bf16;
  const char* name;
  if (!row_type(type, bf16, name)) return refuse(SPTG_ERR_ARG, "rows are f16 or bf16");
  int rc = rows_sizes(rows, cols, top);
  if (rc) return rc;
  if (y_rows < 0 || y_rows > kMaxDim) return refuse(SPTG_ERR_ARG, kDimText);
  if (zero_unnamed != 0 && zero_unnamed != 1) return refuse(SPTG_ERR_ARG, "zero_unnamed must be 0 or 1");
  const bool zeros = zero_unnamed && y_rows > 0 && cols > 0;
  if ((rows == 0 && !zeros) || (cols == 0 && !dweights)) {
    set_config("kernel=none type=%s (empty output)", name, {});
    return SPTG_OK;
  }
  if ((rows > 0 && (!places || (cols > 0 && (!dout || (y_rows > 0 && dweights && !y))))) ||
      (cols > 0 && y_rows > 0 && !dy))
    return refuse(SPTG_ERR_ARG, "null pointer");
  if (dweights && !weights) return refuse(SPTG_ERR_ARG, "dweights belong to weights");
  if (cols > 0 && ((rows > 0 && ldd < cols) || (y_rows > 0 && (lddy < cols || (dweights && ldy < cols)))))
    return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(dout, 2) || off_by(dy, 2) || off_by(y, 2) || off_by(places, 4) || off_by(weights, 4) ||
      off_by(dweights, 4))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  const bool aligned = cols % 8 == 0 && in_pieces(dout, ldd) && in_pieces(dy, lddy) &&
                       (!dweights || in_pieces(y, ldy));
  RowsParams p{};
  p.x = y;
  p.ldx = ldy;
  p.x_rows = y_rows;
  p.places = places;
  p.weights = weights;
  p.dout = dout;
  p.ldd = ldd;
  p.out = dy;
  p.ldo = lddy;
  p.dweights = dweights;
  p.cols = static_cast<int>(cols);
  p.top = top;
  p.entries = rows * top;
  // Rows of dy that no place names. With as many rows as places only entries that were dropped
  // leave some, for blocks of the same launch to find, where what these read is at most as
  // much as zeros for all rows would write (16384 rows of 8 places and 384 columns: 72 us, zeros
  // first 83; cut rows of 385 columns 90 and 100, of 257 columns 85 and 80). Else zeros for all
  // rows go first.
  if (zeros) {
    const int64_t window = std::min<int64_t>(
        aligned ? ZERO_MAX_WINDOW : ZERO_CUT_WINDOW,
        std::max<int64_t>(ZERO_MIN_WINDOW, ceil_div(ceil_div(y_rows, 32), 32) * 32));
    const int64_t blocks = ceil_div(y_rows, window);
    if (y_rows == p.entries && (aligned || cols >= 384) && 2 * blocks <= cols && blocks <= ZERO_MAX_BLOCKS) {
      p.zero_blocks = static_cast<int>(blocks);
      p.zero_window = static_cast<int>(window);
    } else {
      const size_t width = static_cast<size_t>(cols) * 2;
      const cudaError_t e = lddy == cols || y_rows == 1
                                ? cudaMemsetAsync(dy, 0, width * static_cast<size_t>(y_rows), stream)
                                : cudaMemset2DAsync(dy, static_cast<size_t>(lddy) * 2, 0, width,
                                                    static_cast<size_t>(y_rows), stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    }
    if (rows == 0) {
      set_config("kernel=zero-fill type=%s", name, {});
      return SPTG_OK;
    }
  }
  void* args[] = {&p};
  const cudaError_t e = launch_op(combine_rows_grad_variant(bf16, aligned),
                                  dim3(static_cast<unsigned>(rows + p.zero_blocks)), ROWS_THREADS, 0, 1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "combine_rows_grad launch");
  set_config("kernel=combine_grad type=%s aligned=%lld zero_blocks=%lld", name, {aligned, p.zero_blocks});
  return SPTG_OK;
}

// -------------------------------------------- gate, scaled residual and norms
// What a ring may take beside a kernel's own few KB: two rows of three operands of 16384
// elements, or of five of 8192. With cut rows a block keeps 4 KB about their ends, and has a
// thread for each of them: 16 to an operand.
int gate_ring_most(bool cut) { return (cut ? 219 : 223) * 1024; }
int ring_threads_of(int64_t pieces, int per, int ops, bool cut) {
  const int threads = static_cast<int>(ceil_div(ceil_div(pieces, per), 32) * 32);
  return cut ? std::max(threads, static_cast<int>(ceil_div(16 * ops, 32) * 32)) : threads;
}

// Blocks that add up gradients over rows, at most: those of narrow rows are small,
// and an SM holds more of them.
int64_t gate_grad_blocks(int64_t cols) { return 456 * std::max<int64_t>(1, std::min<int64_t>(8, 4096 / std::max<int64_t>(cols, 1))); }

int gate_norm_checks(int64_t rows, int64_t cols, int type, int gate_kind, float alpha, float eps,
                     const sptg_config* cfg, bool& bf16, const char*& name) {
  if (!row_type(type, bf16, name)) return refuse(SPTG_ERR_ARG, "rows are f16 or bf16");
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxCols) return refuse(SPTG_ERR_ARG, kRowText);
  if (gate_kind < SPTG_GATE_NONE || gate_kind > SPTG_GATE_FULL) return refuse(SPTG_ERR_ARG, "unknown kind of gate");
  if (!(eps > 0.0f) || !(eps < INFINITY)) return refuse(SPTG_ERR_ARG, "eps must be positive and finite");
  if (!(alpha > -INFINITY && alpha < INFINITY)) return refuse(SPTG_ERR_ARG, "alpha must be finite");
  if (cfg && (cfg->timeout_ms < 0 || (cfg->inject_stall != 0 && cfg->inject_stall != 1)))
    return refuse(SPTG_ERR_ARG, "timeout_ms must not be negative, inject_stall 0 or 1");
  return SPTG_OK;
}

// Threads of a block that holds a row of `pieces` pieces, `per` to a thread.
int row_threads(int64_t pieces, int per) { return static_cast<int>(ceil_div(ceil_div(pieces, per), 32) * 32); }

// The operands of a ring, in the kernels' order, without those that are null.
GateRing gate_ring(const void* y, int64_t ldy, const void* x, int64_t ldx, const void* dh, int64_t lddh,
                   const void* dv, int64_t lddv, const void* gate, int64_t ldg) {
  GateRing r{};
  const auto add = [&](const void* p, int64_t ld) {
    if (p == nullptr) return;
    r.src[r.ops] = p;
    r.ld[r.ops++] = ld;
  };
  add(y, ldy);
  add(x, ldx);
  add(dh, lddh);
  add(dv, lddv);
  add(gate, ldg);
  return r;
}

void set_ring(GateRing& r, int stages, const DeviceInfo& di, const sptg_config* cfg) {
  r.stages = stages;
  r.error_word = di.error_word;
  r.timeout_ns = cfg && cfg->timeout_ms ? cfg->timeout_ms * 1000000ull : kOpTimeoutNs;
  r.inject_stall = cfg ? cfg->inject_stall : 0;
}

int gate_norm(int64_t rows, int64_t cols, int type, const void* y, int64_t ldy, const void* x, int64_t ldx,
              const void* w1, const void* gate, int gate_kind, int64_t ldg, float alpha, const void* w2,
              float eps, void* h, int64_t ldh, void* v, int64_t ldv, cudaStream_t stream, const sptg_config* cfg) {
  bool bf16;
  const char* name;
  int rc = gate_norm_checks(rows, cols, type, gate_kind, alpha, eps, cfg, bf16, name);
  if (rc) return rc;
  if (rows == 0 || cols == 0) {
    set_config("kernel=none type=%s (empty output)", name, {});
    return SPTG_OK;
  }
  if (!y || !x || !w2 || !h || !v || (gate_kind != SPTG_GATE_NONE && !gate))
    return refuse(SPTG_ERR_ARG, "null pointer");
  if (ldy < cols || ldx < cols || ldh < cols || ldv < cols || (gate_kind == SPTG_GATE_FULL && ldg < cols) ||
      (gate_kind == SPTG_GATE_ROWS && ldg < 1))
    return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
  if (off_by(y, 2) || off_by(x, 2) || off_by(w1, 2) || off_by(w2, 2) || off_by(h, 2) || off_by(v, 2) ||
      (gate_kind != SPTG_GATE_NONE && off_by(gate, 2)))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  const bool vectors = cols % 8 == 0 && in_pieces(y, ldy) && in_pieces(x, ldx) && in_pieces(w1, 0) &&
                       in_pieces(w2, 0) && in_pieces(h, ldh) && in_pieces(v, ldv) &&
                       (gate_kind != SPTG_GATE_COLS || in_pieces(gate, 0)) &&
                       (gate_kind != SPTG_GATE_FULL || in_pieces(gate, ldg));
  const int64_t pieces = cols / 8;
  int kind = GATE_NORM_ANY, threads = GATE_ANY_THREADS;
  if (vectors && pieces <= 2048) {
    kind = pieces <= 512 ? GATE_NORM_1 : GATE_NORM_2;
    threads = row_threads(pieces, kind == GATE_NORM_1 ? 1 : 2);
  } else if (cols <= 16384 - 8) {  // (a piece more where a row's first is cut by a boundary)
    kind = GATE_NORM_SHIFTED;
    threads = row_threads(ceil_div(cols + 7, 8), 2);
  }
  int64_t grid = rows;
  int smem = 0, stages = 0;
  // Rows for several turns of the blocks that the GPU holds: rings, four pieces a thread
  // (16384 rows of 8192: 171 us, a row to a block 211 us; of 4096: 87 and 144 us; 32768 of 512
  // take 36 us either way, and are left to the simpler kernel). Rings of two rows, of three
  // where wide ones leave an SM two blocks (8192 rows of 8192: 87.6 us, with two 90.7 us; 16384
  // of 4096: 89.2 and 87.3 us; with a gate's row as well, 8192 of 5000: 74.0 and 66.6 us).
  if (vectors && pieces > 64 && pieces <= 2048 && rows >= 3 * di.sm_count) {
    const bool full = gate_kind == SPTG_GATE_FULL;
    const void* fn = gate_norm_variant(bf16, GATE_NORM_RING);
    const int ring_threads = row_threads(pieces, 4), ring_stages = cols > 4096 && cols <= 8192 && !full ? 3 : 2;
    const int ring_smem = gate_ring_smem(static_cast<int>(cols), full ? 3 : 2, ring_stages, false);
    Residency res;
    rc = ensure_smem(dev, fn, gate_ring_most(false));
    if (!rc) rc = residency(res, dev, fn, ring_threads, ring_smem);
    if (rc) return rc;
    const int64_t blocks = static_cast<int64_t>(res.blocks) * di.sm_count;
    if (rows >= 3 * blocks) {
      kind = GATE_NORM_RING;
      threads = ring_threads;
      stages = ring_stages;
      smem = ring_smem;
      grid = blocks;
    }
  }
  GateNormParams p{y, x, w1, w2, gate_kind == SPTG_GATE_NONE ? nullptr : gate, ldy, ldx, ldg, h, v, ldh, ldv,
                   rows, static_cast<int>(cols), gate_kind, alpha, eps, {}};
  p.ring = gate_ring(y, ldy, x, ldx, nullptr, 0, nullptr, 0, gate_kind == SPTG_GATE_FULL ? gate : nullptr, ldg);
  set_ring(p.ring, stages, di, cfg);
  void* args[] = {&p};
  const cudaError_t e = launch_op(gate_norm_variant(bf16, kind), dim3(static_cast<unsigned>(grid)), threads, smem,
                                  1, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "gate_add_rms_norm launch");
  set_config("kernel=gate_norm type=%s kind=%lld threads=%lld grid=%lld stages=%lld", name, {kind, threads, grid, stages});
  return SPTG_OK;
}

int64_t gate_grad_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxCols) return 0;
  return 2 * std::min(rows, gate_grad_blocks(cols)) * cols * 4;
}

int gate_norm_grad(int64_t rows, int64_t cols, int type, const void* dh, int64_t lddh, const void* dv,
                   int64_t lddv, const void* y, int64_t ldy, const void* x, int64_t ldx, const void* w1,
                   const void* gate, int gate_kind, int64_t ldg, float alpha, const void* w2, float eps,
                   void* dy, int64_t lddy, void* dx, int64_t lddx, void* dgate, int64_t lddg, void* dw2,
                   void* dw1, int out_type, void* workspace, int64_t workspace_bytes, cudaStream_t stream,
                   const sptg_config* cfg) {
  bool bf16;
  const char* name;
  int rc = gate_norm_checks(rows, cols, type, gate_kind, alpha, eps, cfg, bf16, name);
  if (rc) return rc;
  if (out_type != SPTG_T_F32 && out_type != type)
    return refuse(SPTG_ERR_ARG, "the weights' gradients are f32 or of the rows' type");
  const int out_bytes = out_type == SPTG_T_F32 ? 4 : 2;
  const bool by_row = gate_kind == SPTG_GATE_ROWS, by_col = gate_kind == SPTG_GATE_COLS,
             full = gate_kind == SPTG_GATE_FULL;
  // outputs that exist even where there are no rows, or no columns
  if (cols > 0 && (!dw2 || (w1 && !dw1) || (by_col && !dgate))) return refuse(SPTG_ERR_ARG, "null pointer");
  if (rows > 0 && by_row && !dgate) return refuse(SPTG_ERR_ARG, "null pointer");
  if (rows > 0 && cols > 0) {
    if (!y || !x || !w2 || !dy || !dx || (gate_kind != SPTG_GATE_NONE && (!gate || !dgate)) || !workspace)
      return refuse(SPTG_ERR_ARG, "null pointer");
    if (ldy < cols || ldx < cols || lddy < cols || lddx < cols || (dh && lddh < cols) || (dv && lddv < cols) ||
        (full && (ldg < cols || lddg < cols)) || (by_row && ldg < 1))
      return refuse(SPTG_ERR_ARG, "row pitches must be at least the row lengths");
    if (workspace_bytes < gate_grad_workspace(rows, cols))
      return refuse(SPTG_ERR_ARG, "the workspace is smaller than sptg_gate_add_rms_norm_grad_workspace says");
  }
  if (off_by(y, 2) || off_by(x, 2) || off_by(w1, 2) || off_by(w2, 2) || off_by(dh, 2) || off_by(dv, 2) ||
      off_by(dy, 2) || off_by(dx, 2) || off_by(dw1, out_bytes) || off_by(dw2, out_bytes) ||
      off_by(workspace, 16) || (gate_kind != SPTG_GATE_NONE && (off_by(gate, 2) || off_by(dgate, full ? 2 : out_bytes))))
    return refuse(SPTG_ERR_ALIGN, "a pointer is not aligned to its element type (the workspace: to 16 bytes)");
  int dev = 0;
  DeviceInfo di;
  rc = device_info(di, dev);
  if (rc) return rc;
  if (rows == 0 || cols == 0) {  // empty sums
    cudaError_t e = cudaSuccess;
    if (cols > 0) {
      e = cudaMemsetAsync(dw2, 0, cols * out_bytes, stream);
      if (e == cudaSuccess && w1) e = cudaMemsetAsync(dw1, 0, cols * out_bytes, stream);
      if (e == cudaSuccess && by_col) e = cudaMemsetAsync(dgate, 0, cols * out_bytes, stream);
    } else if (rows > 0 && by_row) {
      e = cudaMemsetAsync(dgate, 0, rows * out_bytes, stream);
    }
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    set_config("kernel=zero-fill type=%s", name, {});
    return SPTG_OK;
  }
  const bool vectors = cols % 8 == 0 && in_pieces(y, ldy) && in_pieces(x, ldx) && in_pieces(w1, 0) &&
                       in_pieces(w2, 0) && in_pieces(dh, lddh) && in_pieces(dv, lddv) && in_pieces(dy, lddy) &&
                       in_pieces(dx, lddx) && (!by_col || in_pieces(gate, 0)) &&
                       (!full || (in_pieces(gate, ldg) && in_pieces(dgate, lddg)));
  // by width and alignment; beyond 8192 columns by a cluster, or element by element
  enum { GATE_GRAD_RING, GATE_GRAD_CUT, GATE_GRAD_WIDE };
  int kind = GATE_GRAD_WIDE, parts = 1, threads = GATE_ANY_THREADS;
  int64_t blocks = 2 * di.sm_count;
  int smem = 0, stages = 0;
  const void* fn = gate_norm_grad_any_variant(bf16);
  const int64_t row_pieces = vectors ? cols / 8 : ceil_div(cols + 7, 8);
  if (cols <= 8192) {
    kind = vectors ? GATE_GRAD_RING : GATE_GRAD_CUT;
    fn = bf16 ? gate_norm_grad_bf16(gate_kind, w1 != nullptr, !vectors)
              : gate_norm_grad_f16(gate_kind, w1 != nullptr, !vectors);
    const int ops = 2 + (dh != nullptr) + (dv != nullptr) + full;
    threads = ring_threads_of(std::min<int64_t>(row_pieces, 1024), 2, ops, !vectors);
    stages = 2;  // (a third row: no faster, and one block an SM less of narrow rows)
    smem = gate_ring_smem(static_cast<int>(cols), ops, stages, !vectors);
    Residency res;
    rc = ensure_smem(dev, fn, gate_ring_most(!vectors));
    if (!rc) rc = residency(res, dev, fn, threads, smem);
    if (rc) return rc;
    blocks = static_cast<int64_t>(res.blocks) * di.sm_count;
  }
  int64_t part_cols = cols;
  if (cols > 8192 && cols <= 8192 * GATE_MAX_PARTS && vectors) {
    // the fewest CTAs that hold a row, and as many clusters as the SMs make
    while (part_cols > 8192) part_cols = ceil_div(cols / 8, parts *= 2) * 8;
    fn = gate_norm_grad_wide_variant(bf16, gate_kind, w1 != nullptr);
    const int ops = 2 + (dh != nullptr) + (dv != nullptr) + full;
    threads = row_threads(part_cols / 8, 2);
    stages = 2;
    smem = gate_ring_smem(static_cast<int>(part_cols), ops, stages, false);
    rc = ensure_smem(dev, fn, gate_ring_most(true));
    if (rc) return rc;
    blocks = di.sm_count / parts;
  }
  blocks = std::min({rows, blocks, gate_grad_blocks(cols)});
  if (kind == GATE_GRAD_CUT && blocks < rows) blocks = std::max<int64_t>(8, blocks / 8 * 8);  // (see RowCut)
  const int out_kind = out_type == SPTG_T_F32 ? OUT_F32 : bf16 ? OUT_BF16 : OUT_F16;
  GateNormGradParams p;
  p.f = GateNormParams{y, x, w1, w2, gate_kind == SPTG_GATE_NONE ? nullptr : gate, ldy, ldx, ldg, nullptr,
                       nullptr, 0, 0, rows, static_cast<int>(cols), gate_kind, alpha, eps, {}};
  p.f.ring = gate_ring(y, ldy, x, ldx, dh, lddh, dv, lddv, full ? gate : nullptr, ldg);
  set_ring(p.f.ring, stages, di, cfg);
  p.dh = dh;
  p.dv = dv;
  p.lddh = lddh;
  p.lddv = lddv;
  p.dy = dy;
  p.dx = dx;
  p.lddy = lddy;
  p.lddx = lddx;
  p.dgate = dgate;
  p.lddg = lddg;
  p.out_kind = out_kind;
  p.parts = parts;
  p.part_cols = static_cast<int>(part_cols);
  p.part = static_cast<float*>(workspace);
  void* args[] = {&p};
  cudaError_t e = launch_op(fn, dim3(static_cast<unsigned>(blocks * parts)), threads, smem,
                            parts, stream, args);
  if (e != cudaSuccess) return cuda_fail(e, "gate_add_rms_norm_grad launch");
  ColumnSumParams c;
  c.part = static_cast<const float*>(workspace);
  c.blocks = static_cast<int>(blocks);
  c.cols = static_cast<int>(cols);
  c.out_kind = out_kind;
  c.dw2 = dw2;
  c.dw1 = w1 ? dw1 : nullptr;
  c.dgate = by_col ? dgate : nullptr;
  c.w1 = w1;
  c.gate = by_col ? gate : nullptr;
  void* column_args[] = {&c};
  e = launch_op(gate_norm_columns_variant(bf16), dim3(static_cast<unsigned>(ceil_div(cols, 32)), by_col || w1 ? 2 : 1),
                1024, 0, 1, stream, column_args);
  if (e != cudaSuccess) return cuda_fail(e, "gate_add_rms_norm_grad columns launch");
  set_config("kernel=gate_norm_grad type=%s kind=%lld threads=%lld grid=%lld stages=%lld parts=%lld", name,
             {kind, threads, blocks, stages, parts});
  return SPTG_OK;
}

}  // namespace

extern "C" {

int sptg_route_experts(int64_t rows, int64_t E, int top, sptg_type type, const void* logits, int64_t ld,
                       const float* bias, int sigmoid, int groups, int top_groups, int group_best,
                       int renormalize, float scale, float* weights, int32_t* experts, void* stream) {
  return guarded([&] {
    return route_experts(rows, E, top, type, logits, ld, bias, sigmoid, groups, top_groups, group_best,
                         renormalize, scale, weights, experts, static_cast<cudaStream_t>(stream));
  });
}

int sptg_route_experts_dlogits(int64_t rows, int64_t E, int top, sptg_type type, const void* logits,
                               int64_t ld, const int32_t* experts, const float* dweights, int sigmoid,
                               int renormalize, float scale, void* dlogits, int64_t ldd, void* stream) {
  return guarded([&] {
    return route_dlogits(rows, E, top, type, logits, ld, experts, dweights, sigmoid, renormalize, scale,
                         dlogits, ldd, static_cast<cudaStream_t>(stream));
  });
}

int sptg_dispatch_rows(int64_t rows, int64_t cols, int top, int64_t E, sptg_type type, const void* x,
                       int64_t ldx, const int32_t* experts, void* sorted, int64_t lds, int32_t* places,
                       int32_t* offsets, void* stream) {
  return guarded([&] {
    return dispatch_rows(rows, cols, top, E, type, x, ldx, experts, sorted, lds, places, offsets,
                         static_cast<cudaStream_t>(stream));
  });
}

int sptg_combine_rows(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type, const void* y,
                      int64_t ldy, const int32_t* places, const float* weights, const void* base,
                      int64_t ldb, void* out, int64_t ldo, void* stream) {
  return guarded([&] {
    return combine_rows(rows, cols, top, y_rows, type, y, ldy, places, weights, base, ldb, out, ldo,
                        static_cast<cudaStream_t>(stream));
  });
}

int sptg_combine_rows_grad(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type,
                           const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* places,
                           const float* weights, void* dy, int64_t lddy, float* dweights, void* stream) {
  return guarded([&] {
    return combine_rows_grad(rows, cols, top, y_rows, type, dout, ldd, y, ldy, places, weights, dy, lddy,
                             dweights, 0, static_cast<cudaStream_t>(stream));
  });
}

int sptg_combine_rows_grad_ex(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type,
                              const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* places,
                              const float* weights, void* dy, int64_t lddy, float* dweights, int zero_unnamed,
                              void* stream) {
  return guarded([&] {
    return combine_rows_grad(rows, cols, top, y_rows, type, dout, ldd, y, ldy, places, weights, dy, lddy,
                             dweights, zero_unnamed, static_cast<cudaStream_t>(stream));
  });
}

int sptg_gate_add_rms_norm(int64_t rows, int64_t cols, sptg_type type, const void* y, int64_t ldy,
                           const void* residual, int64_t ldr, const void* block_weight, const void* gate,
                           sptg_gate gate_kind, int64_t ldg, float alpha, const void* weight, float eps,
                           void* h, int64_t ldh, void* v, int64_t ldv, void* stream, const sptg_config* cfg) {
  return guarded([&] {
    return gate_norm(rows, cols, type, y, ldy, residual, ldr, block_weight, gate, gate_kind, ldg, alpha,
                     weight, eps, h, ldh, v, ldv, static_cast<cudaStream_t>(stream), cfg);
  });
}

int64_t sptg_gate_add_rms_norm_grad_workspace(int64_t rows, int64_t cols) {
  return gate_grad_workspace(rows, cols);
}

int sptg_gate_add_rms_norm_grad(int64_t rows, int64_t cols, sptg_type type, const void* dh, int64_t lddh,
                                const void* dv, int64_t lddv, const void* y, int64_t ldy,
                                const void* residual, int64_t ldr, const void* block_weight,
                                const void* gate, sptg_gate gate_kind, int64_t ldg, float alpha,
                                const void* weight, float eps, void* dy, int64_t lddy, void* dresidual,
                                int64_t lddr, void* dgate, int64_t lddg, void* dweight, void* dblock_weight,
                                sptg_type out_type, void* workspace, int64_t workspace_bytes, void* stream,
                                const sptg_config* cfg) {
  return guarded([&] {
    return gate_norm_grad(rows, cols, type, dh, lddh, dv, lddv, y, ldy, residual, ldr, block_weight, gate,
                          gate_kind, ldg, alpha, weight, eps, dy, lddy, dresidual, lddr, dgate, lddg,
                          dweight, dblock_weight, out_type, workspace, workspace_bytes,
                          static_cast<cudaStream_t>(stream), cfg);
  });
}

}  // extern "C"
