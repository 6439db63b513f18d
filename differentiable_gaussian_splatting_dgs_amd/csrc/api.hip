// C-ABI layer of libgs: argument checks, workspace carving, stream plumbing
// and the status/error strings.  Every check runs on the host before any
// work is enqueued, so a GS_ERR_INVALID_ARG call has launched nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <utility>

#include "../../include/gs.h"
#include "gs_internal.h"

static_assert(GS_MAX_FUSED_VIEWS == gs::kMaxFusedViews, "fused view limit");
static_assert(GS_MAX_PREPROCESS_VIEWS == gs::kMaxPreprocessViews, "preprocess view limit");
static_assert(GS_MAX_COUPLED_VIEWS == gs::kMaxCoupledViews, "coupled view limit");
static_assert(GS_MAX_TILE_BLOCKS == gs::kMaxTileBlocks, "tile block limit");
static_assert(GS_MAX_PARTITION_TILES == gs::kMaxPartitionTiles, "partition tile limit");
static_assert(GS_TYPE_BF16 == gs::kTypeBF16 && GS_TYPE_F16 == gs::kTypeF16 && GS_TYPE_F32 == gs::kTypeF32,
              "storage types");
static_assert(GS_ACT_NONE == gs::kActNone && GS_ACT_RELU == gs::kActRelu && GS_ACT_SILU == gs::kActSilu &&
                  GS_ACT_GELU == gs::kActGelu,
              "activations");
static_assert(GS_MAX_NET_DIM == gs::kMaxNetDim && GS_MAX_NET_GROUPS == gs::kMaxNetGroups, "network limits");
static_assert(GS_MAX_SORT_GROUPS == gs::kMaxSortGroups, "sort limit");
static_assert(GS_MAX_CHOICES == gs::kMaxChoices, "choices limit");
static_assert(GS_ADAMW_BLOCK == gs::kAdamwBlock && GS_MAX_ADAMW_SIZE == gs::kMaxAdamwSize, "adamw limits");

namespace {

thread_local char g_err[512] = "";

gs_status fail(gs_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

gs_status ok() {
  g_err[0] = '\0';
  return GS_OK;
}

gs_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return ok();
  return fail(GS_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int32_t kMaxDim = 65535 * 16;   // tile coordinates are stored in 16 bits

gs_status check_camera(const gs_camera* cam, gs::CamArgs& out) {
  if (cam == nullptr) return fail(GS_ERR_INVALID_ARG, "camera is NULL");
  if (cam->width <= 0 || cam->height <= 0 || cam->width > kMaxDim || cam->height > kMaxDim)
    return fail(GS_ERR_INVALID_ARG, "camera size %dx%d out of range", cam->width, cam->height);
  const float fs[] = {cam->fx, cam->fy, cam->cx, cam->cy, cam->near_z};
  for (float f : fs)
    if (!std::isfinite(f)) return fail(GS_ERR_INVALID_ARG, "camera intrinsics not finite");
  for (int k = 0; k < 9; ++k) out.R[k] = cam->R[k];
  for (int k = 0; k < 3; ++k) {
    out.t[k] = cam->t[k];
    out.campos[k] = cam->campos[k];
  }
  out.fx = cam->fx;
  out.fy = cam->fy;
  out.cx = cam->cx;
  out.cy = cam->cy;
  out.near_z = cam->near_z;
  out.width = cam->width;
  out.height = cam->height;
  out.tiles_x = (cam->width + 15) / 16;
  out.tiles_y = (cam->height + 15) / 16;
  return GS_OK;
}

gs_status check_size(int32_t width, int32_t height) {
  if (width <= 0 || height <= 0 || width > kMaxDim || height > kMaxDim)
    return fail(GS_ERR_INVALID_ARG, "image size %dx%d out of range", width, height);
  return GS_OK;
}

// The split backward's workspace (its size for the image) and segment
// length (a power of two, 64 ... 65536); both ignored without a workspace.
gs_status check_split(const void* ws, size_t ws_bytes, int32_t width, int32_t height, int32_t segment_len,
                      int& seg_shift) {
  seg_shift = 6;
  if (ws == nullptr) return GS_OK;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(GS_ERR_INVALID_ARG, "split_ws not 256-byte aligned");
  const size_t need = gs::raster_split_bytes(width, height);
  if (ws_bytes < need)
    return fail(GS_ERR_INVALID_ARG, "split_ws_bytes = %zu < %zu needed for %dx%d", ws_bytes, need, width, height);
  if (segment_len < 64 || segment_len > 65536 || (segment_len & (segment_len - 1)) != 0)
    return fail(GS_ERR_INVALID_ARG, "segment_len = %d: not a power of two in [64, 65536]", int(segment_len));
  seg_shift = __builtin_ctz(uint32_t(segment_len));
  return GS_OK;
}

#define REQUIRE(cond, ...)                                   \
  do {                                                       \
    if (!(cond)) return fail(GS_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

#define CHECK(expr)                          \
  do {                                       \
    const gs_status s_ = (expr);             \
    if (s_ != GS_OK) return s_;              \
  } while (0)

gs::SsimWindow make_window() {
  gs::SsimWindow w;
  double g[11], s = 0.0;
  for (int k = 0; k < 11; ++k) {
    g[k] = std::exp(-double((k - 5) * (k - 5)) / (2.0 * 1.5 * 1.5));
    s += g[k];
  }
  for (int k = 0; k < 11; ++k) w.g[k] = float(g[k] / s);
  return w;
}

size_t adam_ws_bytes(int64_t n) { return gs::compact_ws_bytes(n); }

// --- network operators ---------------------------------------------------------

gs_status check_net_sizes(int64_t rows, int32_t type) {
  REQUIRE(type >= GS_TYPE_BF16 && type <= GS_TYPE_F32, "type = %d unknown", int(type));
  REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "rows = %lld out of range", (long long)rows);
  return GS_OK;
}

// A row-major matrix argument (rows > 0).
gs_status check_matrix(const char* name, const void* p, int64_t ld, int32_t width, size_t elem) {
  REQUIRE(p != nullptr, "%s is NULL", name);
  REQUIRE(aligned(p, elem), "%s not aligned to its elements", name);
  REQUIRE(ld >= width && ld < (int64_t(1) << 31), "%s: leading dimension %lld for width %d", name, (long long)ld,
          int(width));
  return GS_OK;
}

gs_status check_vector(const char* name, const void* p) {
  REQUIRE(aligned(p, 4), "%s not 4-byte aligned", name);
  return GS_OK;
}

gs_status check_linear(const gs::LinearArgs& a, int64_t rows, int32_t type) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(a.in >= 1 && a.in <= GS_MAX_NET_DIM, "in = %d out of range", int(a.in));
  REQUIRE(a.out >= 1 && a.out <= GS_MAX_NET_DIM, "out = %d out of range", int(a.out));
  REQUIRE(a.act >= GS_ACT_NONE && a.act <= GS_ACT_GELU, "act = %d unknown", int(a.act));
  REQUIRE(a.groups >= 0 && a.groups <= GS_MAX_NET_GROUPS, "num_groups = %d out of range", int(a.groups));
  REQUIRE(gs::linear_fits(rows, a.in, a.out, a.groups), "rows = %lld, in = %d, out = %d pass a launch grid",
          (long long)rows, int(a.in), int(a.out));
  if (a.groups > 0)
    REQUIRE(a.offsets != nullptr && aligned(a.offsets, 8), "offsets NULL or not 8-byte aligned");
  return GS_OK;
}

gs_status linear_fwd(gs::LinearArgs a, int64_t rows, int32_t type, void* stream, const char* where) {
  CHECK(check_linear(a, rows, type));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("x", a.x, a.ldx, a.in, elem));
  CHECK(check_matrix("w", a.w, a.ldw, a.in, elem));
  CHECK(check_matrix("y", a.y, a.ldy, a.out, elem));
  CHECK(check_vector("bias", a.bias));
  if (a.residual != nullptr) CHECK(check_matrix("residual", a.residual, a.ldr, a.out, elem));
  if (a.z != nullptr) CHECK(check_matrix("z", a.z, a.ldz, a.out, elem));
  a.rows = int32_t(rows);
  return hip_status(gs::launch_linear_fwd(type, a, static_cast<hipStream_t>(stream)), where);
}

gs_status linear_bwd(gs::LinearArgs a, int64_t rows, int32_t type, int32_t dw_type, void* ws, size_t ws_bytes,
                     void* stream, const char* where) {
  CHECK(check_linear(a, rows, type));
  const size_t elem = gs::type_bytes(type);
  if (rows > 0) {
    CHECK(check_matrix("dy", a.dy, a.lddy, a.out, elem));
    if (a.act != GS_ACT_NONE) CHECK(check_matrix("z", a.z, a.ldz, a.out, elem));
    if (a.dw != nullptr) CHECK(check_matrix("x", a.x, a.ldx, a.in, elem));
    if (a.dx != nullptr) {
      CHECK(check_matrix("w", a.w, a.ldw, a.in, elem));
      CHECK(check_matrix("dx", a.dx, a.lddx, a.in, elem));
    }
  }
  if (a.dw != nullptr) {
    REQUIRE(dw_type == type || dw_type == GS_TYPE_F32, "dw_type = %d is neither type nor GS_TYPE_F32", int(dw_type));
    REQUIRE(aligned(a.dw, gs::type_bytes(dw_type)), "dw not aligned to its elements");
  }
  CHECK(check_vector("db", a.db));
  REQUIRE(ws != nullptr && aligned(ws, 256), "workspace NULL or not 256-byte aligned");
  const size_t need = gs::linear_bwd_ws_bytes(type, rows, a.in, a.out, a.groups, a.act);
  REQUIRE(ws_bytes >= need, "workspace_bytes = %zu < %zu needed", ws_bytes, need);
  a.rows = int32_t(rows);
  a.dw_f32 = dw_type == GS_TYPE_F32;
  return hip_status(gs::launch_linear_bwd(type, a, ws, static_cast<hipStream_t>(stream)), where);
}

}  // namespace

// The scratch of gs_sparse_adam_noalloc.  In host code `scratch` names a
// host-side stand-in, not device memory: kernels get the address that
// hipGetSymbolAddress returns for the current device (each device holds its
// own copy), taken once per device and kept in g_scratch_ptr.
static __device__ __align__(256) unsigned char scratch[GS_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxScratchDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxScratchDevices] = {};

// The device address of `scratch` on the current device (looked up on the
// first call on that device).
gs_status scratch_address(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e, "gs_sparse_adam_noalloc (hipGetDevice)");
  if (dev < 0 || dev >= kMaxScratchDevices)
    return fail(GS_ERR_HIP, "gs_sparse_adam_noalloc: device %d beyond the %d the library tracks", dev,
                kMaxScratchDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_status(e, "gs_sparse_adam_noalloc (hipGetSymbolAddress)");
    if (p == nullptr) return fail(GS_ERR_HIP, "gs_sparse_adam_noalloc: NULL scratch address");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return GS_OK;
}

gs_status check_ids(const void* ids, int32_t id_bytes, int64_t n) {
  REQUIRE(id_bytes == 4 || id_bytes == 8, "id_bytes = %d: 4 or 8 expected", int(id_bytes));
  REQUIRE(n == 0 || (ids != nullptr && aligned(ids, size_t(id_bytes))), "ids NULL or not aligned to its elements");
  return GS_OK;
}

gs_status check_sort_sizes(int64_t n, int64_t num_groups) {
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(num_groups >= 1 && num_groups <= GS_MAX_SORT_GROUPS, "num_groups = %lld out of range",
          (long long)num_groups);
  return GS_OK;
}

gs_status check_gate(const gs::GateArgs& a, int64_t rows, int32_t type) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(a.groups >= 1 && a.groups <= GS_MAX_NET_GROUPS, "groups = %d out of range", int(a.groups));
  REQUIRE(a.k >= 1 && a.k <= std::min(a.groups, GS_MAX_CHOICES), "k = %d out of range", int(a.k));
  if (rows == 0) return GS_OK;
  REQUIRE(a.ids != nullptr && a.weights != nullptr, "ids / weights NULL");
  CHECK(check_vector("ids", a.ids));
  CHECK(check_vector("weights", a.weights));
  return GS_OK;
}

gs_status check_route(const gs::RouteArgs& a, int64_t rows, int32_t type) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(a.k >= 1 && a.k <= GS_MAX_CHOICES, "k = %d out of range", int(a.k));
  REQUIRE(rows * a.k < (int64_t(1) << 31), "rows = %lld with k = %d out of range", (long long)rows, int(a.k));
  REQUIRE(a.width >= 1 && a.width <= GS_MAX_NET_DIM, "width = %d out of range", int(a.width));
  if (rows == 0) return GS_OK;
  REQUIRE(a.place != nullptr && aligned(a.place, 4), "place NULL or not 4-byte aligned");
  CHECK(check_vector("weights", a.weights));
  if (a.residual != nullptr) {
    CHECK(check_matrix("residual", a.residual, a.ldr, a.width, gs::type_bytes(type)));
    REQUIRE(a.residual != a.y || a.ldr == a.ldy, "in place with leading dimensions %lld and %lld", (long long)a.ldr,
            (long long)a.ldy);
  }
  return GS_OK;
}

gs_status check_embedding(int64_t rows, int64_t num_rows, int32_t width, int32_t type) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(num_rows >= 1 && num_rows <= GS_MAX_SORT_GROUPS, "num_rows = %lld out of range", (long long)num_rows);
  REQUIRE(width >= 1 && width <= GS_MAX_NET_DIM, "width = %d out of range", int(width));
  return GS_OK;
}

}  // namespace

extern "C" {

const char* gs_status_string(int status) {
  switch (status) {
    case GS_OK: return "GS_OK";
    case GS_ERR_INVALID_ARG: return "GS_ERR_INVALID_ARG: invalid argument";
    case GS_ERR_CAPACITY: return "GS_ERR_CAPACITY: pair capacity exceeded";
    case GS_ERR_HIP: return "GS_ERR_HIP: HIP runtime error";
    default: return "unknown gs_status";
  }
}

const char* gs_last_error(void) { return g_err; }

int gs_version(void) { return 1; }

gs_status gs_workspace_size(gs_op op, int64_t n, int32_t width, int32_t height, int64_t pair_capacity,
                            size_t* bytes) {
  REQUIRE(bytes != nullptr, "bytes is NULL");
  switch (op) {
    case GS_OP_PREPROCESS:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      *bytes = gs::preprocess_ws_bytes(n);
      return ok();
    case GS_OP_BIN_SORT:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      REQUIRE(pair_capacity >= 0 && pair_capacity < (int64_t(1) << 31), "pair_capacity out of range");
      *bytes = gs::binsort_ws_bytes(n, pair_capacity);
      return ok();
    case GS_OP_LOSS:
      CHECK(check_size(width, height));
      *bytes = gs::loss_ws_bytes(width, height);
      return ok();
    case GS_OP_SPARSE_ADAM:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      *bytes = adam_ws_bytes(n);
      return ok();
    case GS_OP_RASTER:
      CHECK(check_size(width, height));
      *bytes = gs::raster_split_bytes(width, height);
      return ok();
    case GS_OP_PREPROCESS_VIEWS:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      REQUIRE(width >= 1 && width <= GS_MAX_PREPROCESS_VIEWS, "num_views = %d out of range", width);
      *bytes = gs::preprocess_views_ws_bytes(n, width);
      return ok();
    case GS_OP_LAYER_NORM_BWD:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "rows = %lld out of range", (long long)n);
      REQUIRE(width >= 1 && width <= GS_MAX_NET_DIM, "width = %d out of range", width);
      *bytes = gs::layer_norm_ws_bytes(n, width);
      return ok();
    case GS_OP_DENSIFY:
      REQUIRE(n >= 0 && n < (int64_t(1) << 30), "n = %lld out of range", (long long)n);
      *bytes = gs::densify_ws_bytes(n);
      return ok();
    case GS_OP_PACK:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      REQUIRE(width >= 1 && width <= GS_MAX_TILE_BLOCKS, "num_blocks = %d out of range", width);
      *bytes = gs::pack_ws_bytes(n, width);
      return ok();
    case GS_OP_VIEW_OVERLAP:
      REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
      REQUIRE(width >= 0 && width <= GS_MAX_COUPLED_VIEWS, "num_views = %d out of range", width);
      *bytes = gs::coupling_ws_bytes(n, width);
      return ok();
  }
  return fail(GS_ERR_INVALID_ARG, "unknown op %d", int(op));
}

gs_status gs_preprocess(const float* params, int64_t n, int64_t ld, const gs_camera* cam, float* proj,
                        float* proj_bin, int32_t* vis_idx, int64_t* vis_count, uint8_t* union_flags, void* workspace,
                        size_t workspace_bytes, void* stream) {
  gs::CamArgs c;
  CHECK(check_camera(cam, c));
  REQUIRE(n >= 0 && n < GS_MAX_PLANE_ROWS, "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(vis_count != nullptr, "vis_count is NULL");
  if (n > 0) {
    REQUIRE(params && proj && vis_idx, "NULL array");
    REQUIRE(aligned(proj, 16) && aligned(params, 4) && aligned(vis_idx, 4), "misaligned array");
  }
  REQUIRE(proj_bin == nullptr || aligned(proj_bin, 16), "proj_bin not 16-byte aligned");
  REQUIRE(union_flags == nullptr || aligned(union_flags, 16), "union_flags not 16-byte aligned");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::preprocess_ws_bytes(n), "workspace too small");
  return hip_status(gs::launch_preprocess(params, n, ld, c, proj, proj_bin, vis_idx, vis_count, union_flags,
                                          workspace, static_cast<hipStream_t>(stream)),
                    "gs_preprocess");
}

gs_status gs_preprocess_views(const float* params, int64_t n, int64_t ld, const gs_camera* cams, int32_t num_views,
                              float* const* proj, float* const* proj_bin, int32_t* const* vis_idx,
                              int64_t* vis_count, uint8_t* union_flags, int32_t max_workgroups, void* workspace,
                              size_t workspace_bytes, void* stream) {
  REQUIRE(num_views >= 1 && num_views <= GS_MAX_PREPROCESS_VIEWS, "num_views = %d outside [1, %d]", int(num_views),
          GS_MAX_PREPROCESS_VIEWS);
  REQUIRE(cams != nullptr && proj != nullptr && vis_idx != nullptr, "cams / proj / vis_idx NULL");
  gs::CamArgs c[gs::kMaxPreprocessViews];
  for (int32_t w = 0; w < num_views; ++w) CHECK(check_camera(cams + w, c[w]));
  REQUIRE(n >= 0 && n < GS_MAX_PLANE_ROWS, "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(vis_count != nullptr && aligned(vis_count, 8), "vis_count NULL or misaligned");
  if (n > 0) {
    REQUIRE(params != nullptr && aligned(params, 4), "params NULL or misaligned");
    for (int32_t w = 0; w < num_views; ++w) {
      REQUIRE(proj[w] != nullptr && aligned(proj[w], 16), "proj[%d] NULL or not 16-byte aligned", int(w));
      REQUIRE(vis_idx[w] != nullptr && aligned(vis_idx[w], 4), "vis_idx[%d] NULL or misaligned", int(w));
    }
  }
  if (proj_bin != nullptr)
    for (int32_t w = 0; w < num_views; ++w)
      REQUIRE(proj_bin[w] == nullptr || aligned(proj_bin[w], 16), "proj_bin[%d] not 16-byte aligned", int(w));
  REQUIRE(union_flags == nullptr || aligned(union_flags, 16), "union_flags not 16-byte aligned");
  REQUIRE(max_workgroups >= 0, "max_workgroups = %d < 0", int(max_workgroups));
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::preprocess_views_ws_bytes(n, num_views), "workspace too small");
  return hip_status(gs::launch_preprocess_views(params, n, ld, c, num_views, proj, proj_bin, vis_idx, vis_count,
                                                union_flags, max_workgroups, workspace,
                                                static_cast<hipStream_t>(stream)),
                    "gs_preprocess_views");
}

gs_status gs_bin_sort(const float* proj, const float* proj_bin, int64_t n, const int32_t* vis_idx,
                      const int64_t* vis_count,
                      int32_t width, int32_t height, uint64_t* keys, int32_t* vals, int64_t pair_capacity,
                      int64_t* num_pairs, uint32_t* tile_ranges, uint32_t* tile_order, void* workspace,
                      size_t workspace_bytes, void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(pair_capacity >= 0 && pair_capacity < (int64_t(1) << 31), "pair_capacity out of range");
  REQUIRE(vis_count != nullptr && num_pairs != nullptr && tile_ranges != nullptr, "NULL argument");
  if (n > 0) REQUIRE(proj && vis_idx && aligned(proj, 16), "NULL or misaligned proj / vis_idx");
  REQUIRE(proj_bin == nullptr || aligned(proj_bin, 16), "proj_bin not 16-byte aligned");
  if (pair_capacity > 0)
    REQUIRE(vals && (keys ? aligned(keys, 8) : gs::binsort_keys_optional((width + 15) / 16, (height + 15) / 16)),
            "NULL or misaligned keys / vals (keys may be NULL only up to 256 x 256 tiles)");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::binsort_ws_bytes(n, pair_capacity), "workspace too small");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int32_t TX = (width + 15) / 16, TY = (height + 15) / 16;
  hipError_t e =
      gs::launch_binsort_stage1(proj, proj_bin, n, vis_idx, vis_count, TX, TY, nullptr, workspace, pair_capacity,
                                st);
  if (e != hipSuccess) return hip_status(e, "gs_bin_sort (depth sort)");
  int64_t M = 0;
  e = hipMemcpyAsync(&M, gs::binsort_count_ptr(workspace, n, pair_capacity), sizeof(int64_t), hipMemcpyDeviceToHost,
                     st);
  if (e == hipSuccess) e = hipStreamSynchronize(st);
  if (e != hipSuccess) return hip_status(e, "gs_bin_sort (pair count)");
  *num_pairs = M;
  if (M > pair_capacity)
    return fail(GS_ERR_CAPACITY, "%lld pairs > capacity %lld", (long long)M, (long long)pair_capacity);
  e = gs::launch_binsort_stage2(proj, n, vis_idx, vis_count, M, TX, TY, keys, vals, tile_ranges, tile_order,
                                workspace, pair_capacity, st);
  return hip_status(e, "gs_bin_sort");
}

gs_status gs_bin_sort_async(const float* proj, const float* proj_bin, int64_t n, const int32_t* vis_idx,
                            const int64_t* vis_count,
                            int32_t width, int32_t height, uint64_t* keys, int32_t* vals, int64_t pair_capacity,
                            int64_t* num_pairs_dev, uint32_t* tile_ranges, uint32_t* tile_order, void* workspace,
                            size_t workspace_bytes, int32_t part, void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(part == GS_BIN_ALL || part == GS_BIN_DEPTH || part == GS_BIN_PAIRS, "part = %d is not a binning part",
          int(part));
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(pair_capacity >= 0 && pair_capacity < (int64_t(1) << 31), "pair_capacity out of range");
  REQUIRE(vis_count != nullptr && num_pairs_dev != nullptr && tile_ranges != nullptr, "NULL argument");
  REQUIRE(aligned(num_pairs_dev, 8), "misaligned num_pairs_dev");
  if (n > 0) REQUIRE(proj && vis_idx && aligned(proj, 16), "NULL or misaligned proj / vis_idx");
  REQUIRE(proj_bin == nullptr || aligned(proj_bin, 16), "proj_bin not 16-byte aligned");
  if (pair_capacity > 0)
    REQUIRE(vals && (keys ? aligned(keys, 8) : gs::binsort_keys_optional((width + 15) / 16, (height + 15) / 16)),
            "NULL or misaligned keys / vals (keys may be NULL only up to 256 x 256 tiles)");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::binsort_ws_bytes(n, pair_capacity), "workspace too small");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int32_t TX = (width + 15) / 16, TY = (height + 15) / 16;
  hipError_t e = hipSuccess;
  if (part != GS_BIN_PAIRS) {
    e = gs::launch_binsort_stage1(proj, proj_bin, n, vis_idx, vis_count, TX, TY, num_pairs_dev, workspace,
                                  pair_capacity, st);
    if (e != hipSuccess) return hip_status(e, "gs_bin_sort_async (depth sort)");
  }
  if (part != GS_BIN_DEPTH)
    e = gs::launch_binsort_stage2(proj, n, vis_idx, vis_count, -1, TX, TY, keys, vals, tile_ranges, tile_order,
                                  workspace, pair_capacity, st);
  return hip_status(e, "gs_bin_sort_async");
}

gs_status gs_render_fwd(const float* proj, int64_t n, const int32_t* vals, const uint32_t* tile_ranges,
                        const uint32_t* tile_order, int64_t num_pairs, int32_t width, int32_t height, float* image,
                        float* T_final, uint32_t* last, uint32_t* tile_processed, void* split_ws,
                        size_t split_ws_bytes, int32_t segment_len, void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(n >= 0 && num_pairs >= 0 && num_pairs < (int64_t(1) << 31), "n / num_pairs out of range");
  REQUIRE(tile_ranges && image && T_final && last, "NULL output or tile_ranges");
  if (num_pairs > 0) REQUIRE(proj && vals && aligned(proj, 16), "NULL or misaligned proj / vals");
  int seg_shift = 0;
  CHECK(check_split(split_ws, split_ws_bytes, width, height, segment_len, seg_shift));
  return hip_status(gs::launch_render_fwd(proj, vals, tile_ranges, tile_order, num_pairs, width, height, image,
                                          T_final, last, tile_processed, split_ws, seg_shift,
                                          static_cast<hipStream_t>(stream)),
                    "gs_render_fwd");
}

gs_status gs_loss(const float* image, const float* target, int32_t width, int32_t height, float w_l1,
                  float w_ssim, float* loss, float* dL_dimage, void* workspace, size_t workspace_bytes,
                  void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(image && target && loss && dL_dimage, "NULL argument");
  REQUIRE(std::isfinite(w_l1) && std::isfinite(w_ssim), "loss weights not finite");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::loss_ws_bytes(width, height), "workspace too small");
  static const gs::SsimWindow win = make_window();
  return hip_status(gs::launch_loss(image, target, width, height, w_l1, w_ssim, win, loss, dL_dimage, workspace,
                                    static_cast<hipStream_t>(stream)),
                    "gs_loss");
}

gs_status gs_render_bwd(const float* proj, int64_t n, const int32_t* vals, const uint32_t* tile_ranges,
                        const uint32_t* tile_order, int64_t num_pairs, int32_t width, int32_t height,
                        const float* T_final, const uint32_t* last, const float* dL_dimage, float* grad2d,
                        const void* split_ws, size_t split_ws_bytes, int32_t segment_len,
                        const gs_param_grads* param_grads, uint64_t* visits, uint8_t* touched,
                        int32_t touched_slot, void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(num_pairs >= 0 && num_pairs < (int64_t(1) << 31), "num_pairs out of range");
  REQUIRE(tile_ranges && T_final && last && dL_dimage, "NULL argument");
  if (num_pairs > 0 || (param_grads != nullptr && n > 0)) {
    REQUIRE(grad2d != nullptr && aligned(grad2d, 16), "grad2d NULL or not 16-byte aligned");
  }
  if (num_pairs > 0) REQUIRE(proj && vals && aligned(proj, 16), "NULL or misaligned proj / vals");
  REQUIRE(visits == nullptr || aligned(visits, 8), "visits not 8-byte aligned");
  if (touched != nullptr) {
    REQUIRE(aligned(touched, 16), "touched not 16-byte aligned");
    REQUIRE(touched_slot >= 0 && touched_slot < GS_TOUCHED_SLOTS, "touched_slot = %d out of range", touched_slot);
    REQUIRE(param_grads == nullptr, "touched with param_grads (the screen-space rows are consumed in the call)");
  }
  int seg_shift = 0;
  CHECK(check_split(split_ws, split_ws_bytes, width, height, segment_len, seg_shift));
  gs::CamArgs c{};
  if (param_grads != nullptr) {
    CHECK(check_camera(param_grads->cam, c));
    REQUIRE(c.width == width && c.height == height, "param_grads->cam is %dx%d, the image %dx%d", c.width, c.height,
            width, height);
    REQUIRE(n < GS_MAX_PLANE_ROWS, "n = %lld out of range with param_grads", (long long)n);
    REQUIRE(param_grads->ld >= n, "param_grads->ld < n");
    REQUIRE(param_grads->vis_count != nullptr, "param_grads->vis_count is NULL");
    if (n > 0)
      REQUIRE(param_grads->params && param_grads->vis_idx && param_grads->grads, "NULL array in param_grads");
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = gs::launch_render_bwd(proj, vals, tile_ranges, tile_order, num_pairs, width, height, T_final, last,
                                       dL_dimage, grad2d, touched != nullptr ? touched + touched_slot : nullptr,
                                       split_ws, seg_shift, visits, st);
  if (e == hipSuccess && param_grads != nullptr)
    e = gs::launch_project_bwd(param_grads->params, n, param_grads->ld, c, param_grads->vis_idx,
                               param_grads->vis_count, grad2d, param_grads->grads, st);
  return hip_status(e, "gs_render_bwd");
}

gs_status gs_project_bwd(const float* params, int64_t n, int64_t ld, const gs_camera* cam, const int32_t* vis_idx,
                         const int64_t* vis_count, float* grad2d, float* grads, void* stream) {
  gs::CamArgs c;
  CHECK(check_camera(cam, c));
  REQUIRE(n >= 0 && n < GS_MAX_PLANE_ROWS, "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(vis_count != nullptr, "vis_count is NULL");
  if (n > 0) {
    REQUIRE(params && vis_idx && grad2d && grads, "NULL array");
    REQUIRE(aligned(grad2d, 16), "grad2d not 16-byte aligned");
  }
  return hip_status(gs::launch_project_bwd(params, n, ld, c, vis_idx, vis_count, grad2d, grads,
                                           static_cast<hipStream_t>(stream)),
                    "gs_project_bwd");
}

gs_status gs_sparse_adam(float* params, float* grads, float* m, float* v, int64_t n, int64_t ld,
                         uint8_t* union_flags, int32_t* union_idx, int64_t* union_count, float lr, float beta1,
                         float beta2, float eps, float bias_c1, float bias_c2, void* workspace,
                         size_t workspace_bytes, void* stream) {
  REQUIRE(n >= 0 && n < GS_MAX_PLANE_ROWS, "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(union_count != nullptr, "union_count is NULL");
  if (n > 0) {
    REQUIRE(params && grads && m && v && union_flags && union_idx, "NULL array");
    REQUIRE(aligned(union_flags, 16), "union_flags not 16-byte aligned");
  }
  REQUIRE(std::isfinite(lr) && std::isfinite(beta1) && std::isfinite(beta2) && std::isfinite(eps), "non-finite scalar");
  REQUIRE(bias_c1 > 0.0f && bias_c2 > 0.0f, "bias corrections must be > 0");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= adam_ws_bytes(n), "workspace too small");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = gs::launch_compact(union_flags, n, union_idx, union_count, true, workspace, st);
  if (e == hipSuccess)
    e = gs::launch_sparse_adam(params, grads, m, v, n, ld, union_idx, union_count, lr, beta1, beta2, eps, bias_c1,
                               bias_c2, st);
  return hip_status(e, "gs_sparse_adam");
}

gs_status gs_sparse_adam_noalloc(float* params, float* grads, float* m, float* v, int64_t n, int64_t ld,
                                 uint8_t* union_flags, int32_t* union_idx, int64_t* union_count, float lr,
                                 float beta1, float beta2, float eps, float bias_c1, float bias_c2, void* stream) {
  REQUIRE(n >= 0 && n <= GS_NOALLOC_MAX_N, "n = %lld outside [0, %lld]: the union compaction needs %zu scratch "
          "bytes, the allocation-free entry holds %zu", (long long)n, (long long)GS_NOALLOC_MAX_N,
          adam_ws_bytes(n), size_t(GS_NOALLOC_SCRATCH_BYTES));
  REQUIRE(adam_ws_bytes(n) <= size_t(GS_NOALLOC_SCRATCH_BYTES), "n = %lld: scratch too small", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(union_count != nullptr, "union_count is NULL");
  if (n > 0) {
    REQUIRE(params && grads && m && v && union_flags && union_idx, "NULL array");
    REQUIRE(aligned(union_flags, 16), "union_flags not 16-byte aligned");
  }
  REQUIRE(std::isfinite(lr) && std::isfinite(beta1) && std::isfinite(beta2) && std::isfinite(eps), "non-finite scalar");
  REQUIRE(bias_c1 > 0.0f && bias_c2 > 0.0f, "bias corrections must be > 0");
  static_assert(GS_NOALLOC_SCRATCH_BYTES % 256 == 0, "scratch size");
  void* ws = nullptr;
  CHECK(scratch_address(&ws));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // (k_count writes every block count k_scan_counts and k_write read)
  hipError_t e = gs::launch_compact(union_flags, n, union_idx, union_count, true, ws, st);
  if (e == hipSuccess)
    e = gs::launch_sparse_adam(params, grads, m, v, n, ld, union_idx, union_count, lr, beta1, beta2, eps, bias_c1,
                               bias_c2, st);
  return hip_status(e, "gs_sparse_adam_noalloc");
}

gs_status gs_project_bwd_adam(float* params, float* grads, float* m, float* v, int64_t n, int64_t ld,
                              const gs_camera* cams, int32_t num_views, float* const* grad2d, uint8_t* touched,
                              uint8_t* union_flags, int32_t* union_idx, int64_t* union_count,
                              const gs_camera* next_cam,
                              float* next_proj, float* next_proj_bin, uint8_t* next_flags, float lr, float beta1,
                              float beta2, float eps, float bias_c1, float bias_c2, void* workspace,
                              size_t workspace_bytes, void* stream) {
  REQUIRE(num_views >= 0 && num_views <= GS_MAX_FUSED_VIEWS, "num_views = %d outside [0, %d]", int(num_views),
          GS_MAX_FUSED_VIEWS);
  REQUIRE(num_views == 0 || (cams != nullptr && grad2d != nullptr), "cams / grad2d NULL");
  REQUIRE(touched == nullptr || aligned(touched, 16), "touched not 16-byte aligned");
  gs::FusedViews fv{};
  fv.count = num_views;
  fv.touched = touched;
  for (int32_t w = 0; w < num_views; ++w) {
    CHECK(check_camera(cams + w, fv.cam[w]));
    fv.grad2d[w] = grad2d[w];
  }
  REQUIRE(n >= 0 && n < GS_MAX_PLANE_ROWS, "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n, "ld < n");
  REQUIRE(union_count != nullptr, "union_count is NULL");
  if (n > 0) {
    REQUIRE(params && m && v && union_flags && union_idx, "NULL array");
    REQUIRE(aligned(union_flags, 16), "union_flags not 16-byte aligned");
    for (int32_t w = 0; w < num_views; ++w)
      REQUIRE(fv.grad2d[w] != nullptr && aligned(fv.grad2d[w], 16), "grad2d[%d] NULL or not 16-byte aligned",
              int(w));
  }
  REQUIRE(std::isfinite(lr) && std::isfinite(beta1) && std::isfinite(beta2) && std::isfinite(eps), "non-finite scalar");
  REQUIRE(bias_c1 > 0.0f && bias_c2 > 0.0f, "bias corrections must be > 0");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= adam_ws_bytes(n), "workspace too small");
  REQUIRE((next_cam == nullptr) == (next_proj == nullptr) && (next_cam == nullptr) == (next_flags == nullptr),
          "next_cam, next_proj and next_flags: all NULL or none");
  REQUIRE(next_cam != nullptr || next_proj_bin == nullptr, "next_proj_bin given without next_proj");
  if (next_cam != nullptr) {
    CHECK(check_camera(next_cam, fv.next));
    REQUIRE(aligned(next_proj, 16), "next_proj not 16-byte aligned");
    REQUIRE(next_proj_bin == nullptr || aligned(next_proj_bin, 16), "next_proj_bin not 16-byte aligned");
    fv.next_proj = next_proj;
    fv.next_bin = next_proj_bin;
    fv.next_flags = next_flags;
    fv.union_flags = union_flags;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = gs::launch_compact(union_flags, n, union_idx, union_count, true, workspace, st);
  if (e == hipSuccess)
    e = gs::launch_project_adam(params, grads, m, v, n, ld, fv, union_idx, union_count, lr, beta1, beta2, eps,
                                bias_c1, bias_c2, st);
  return hip_status(e, "gs_project_bwd_adam");
}

gs_status gs_visible_list(uint8_t* flags, int64_t n, int32_t* vis_idx, int64_t* vis_count, void* workspace,
                          size_t workspace_bytes, void* stream) {
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(vis_count != nullptr, "vis_count is NULL");
  if (n > 0) REQUIRE(flags && vis_idx && aligned(flags, 16), "NULL or misaligned flags / vis_idx");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::compact_ws_bytes(n), "workspace too small");
  return hip_status(gs::launch_compact(flags, n, vis_idx, vis_count, true, workspace,
                                       static_cast<hipStream_t>(stream)),
                    "gs_visible_list");
}

gs_status gs_view_overlap(const int32_t* lists, int64_t ld, const int64_t* counts, int32_t num_views, int64_t n,
                          int64_t* inter, double* weights, void* workspace, size_t workspace_bytes, void* stream) {
  REQUIRE(num_views >= 0 && num_views <= GS_MAX_COUPLED_VIEWS, "num_views = %d out of range", num_views);
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(ld >= 1, "ld = %lld < 1", (long long)ld);
  if (num_views == 0) return ok();
  REQUIRE(lists != nullptr && counts != nullptr, "lists or counts is NULL");
  REQUIRE(aligned(counts, 8), "counts not 8-byte aligned");
  REQUIRE(inter != nullptr && aligned(inter, 8), "inter NULL or not 8-byte aligned");
  REQUIRE(weights == nullptr || aligned(weights, 8), "weights not 8-byte aligned");
  REQUIRE(aligned(lists, 4), "lists not 4-byte aligned");
  const size_t need = gs::coupling_ws_bytes(n, num_views);
  if (need > 0) {
    REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
    REQUIRE(workspace_bytes >= need, "workspace too small (%zu < %zu)", workspace_bytes, need);
  }
  return hip_status(gs::launch_view_overlap(lists, ld, counts, num_views, n, inter, weights, workspace,
                                            static_cast<hipStream_t>(stream)),
                    "gs_view_overlap");
}

gs_status gs_view_priority(const double* weights, int32_t num_views, const int32_t* prev, int32_t num_prev,
                           double* score, void* stream) {
  REQUIRE(num_views >= 0 && num_views <= GS_MAX_COUPLED_VIEWS, "num_views = %d out of range", num_views);
  REQUIRE(num_prev >= 0, "num_prev = %d < 0", num_prev);
  if (num_views == 0) return ok();
  REQUIRE(weights != nullptr && aligned(weights, 8), "weights NULL or not 8-byte aligned");
  REQUIRE(score != nullptr && aligned(score, 8), "score NULL or not 8-byte aligned");
  REQUIRE(num_prev == 0 || prev != nullptr, "prev is NULL");
  return hip_status(gs::launch_view_priority(weights, num_views, prev, num_prev, score,
                                             static_cast<hipStream_t>(stream)),
                    "gs_view_priority");
}

gs_status gs_tile_partition(const uint32_t* cost, int32_t num_tiles, int32_t num_blocks, int32_t* bounds,
                            void* stream) {
  REQUIRE(num_tiles >= 1 && num_tiles <= GS_MAX_PARTITION_TILES, "num_tiles = %d out of range", num_tiles);
  REQUIRE(num_blocks >= 1 && num_blocks <= GS_MAX_TILE_BLOCKS, "num_blocks = %d out of range", num_blocks);
  REQUIRE(cost != nullptr && aligned(cost, 4), "cost NULL or misaligned");
  REQUIRE(bounds != nullptr && aligned(bounds, 4), "bounds NULL or misaligned");
  return hip_status(gs::launch_tile_partition(cost, num_tiles, num_blocks, bounds, static_cast<hipStream_t>(stream)),
                    "gs_tile_partition");
}

gs_status gs_pack_records(const float* proj, int64_t n, const int32_t* vis_idx, const int64_t* vis_count,
                          int32_t width, int32_t height, const int32_t* bounds, int32_t num_blocks,
                          int64_t capacity, int64_t* send_offsets, int32_t* send_idx, float* send_rec,
                          void* workspace, size_t workspace_bytes, void* stream) {
  CHECK(check_size(width, height));
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(num_blocks >= 1 && num_blocks <= GS_MAX_TILE_BLOCKS, "num_blocks = %d out of range", num_blocks);
  REQUIRE(capacity >= 0 && capacity < (int64_t(1) << 40), "capacity out of range");
  REQUIRE(vis_count != nullptr && aligned(vis_count, 8), "vis_count NULL or misaligned");
  REQUIRE(bounds != nullptr && aligned(bounds, 4), "bounds NULL or misaligned");
  REQUIRE(send_offsets != nullptr && aligned(send_offsets, 8), "send_offsets NULL or misaligned");
  if (n > 0) REQUIRE(proj != nullptr && aligned(proj, 16) && vis_idx != nullptr, "NULL or misaligned proj / vis_idx");
  if (capacity > 0) {
    REQUIRE(send_idx != nullptr, "send_idx is NULL");
    REQUIRE(send_rec == nullptr || aligned(send_rec, 16), "send_rec not 16-byte aligned");
  }
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::pack_ws_bytes(n, num_blocks), "workspace too small");
  return hip_status(gs::launch_pack_records(proj, n, vis_idx, vis_count, (width + 15) / 16, bounds, num_blocks,
                                            capacity, send_offsets, send_idx, send_rec, workspace,
                                            static_cast<hipStream_t>(stream)),
                    "gs_pack_records");
}

gs_status gs_unpack_grads(const float* recv_grad, const int64_t* send_offsets, const int32_t* send_idx,
                          int32_t num_blocks, int64_t capacity, float* grad2d, int64_t n, void* stream) {
  REQUIRE(num_blocks >= 1 && num_blocks <= GS_MAX_TILE_BLOCKS, "num_blocks = %d out of range", num_blocks);
  REQUIRE(capacity >= 0 && capacity < (int64_t(1) << 40), "capacity out of range");
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(send_offsets != nullptr && aligned(send_offsets, 8), "send_offsets NULL or misaligned");
  if (capacity > 0)
    REQUIRE(recv_grad != nullptr && aligned(recv_grad, 16) && send_idx != nullptr,
            "NULL or misaligned recv_grad / send_idx");
  if (n > 0) REQUIRE(grad2d != nullptr && aligned(grad2d, 16), "grad2d NULL or not 16-byte aligned");
  if (capacity == 0 || n == 0) return ok();
  return hip_status(gs::launch_unpack_grads(recv_grad, send_offsets, send_idx, num_blocks, capacity, grad2d, n,
                                            static_cast<hipStream_t>(stream)),
                    "gs_unpack_grads");
}

gs_status gs_densify_stats(const float* grad2d, const int32_t* vis_idx, const int64_t* vis_count, int64_t n,
                           float* accum, int32_t* denom, void* stream) {
  REQUIRE(n >= 0 && n < (int64_t(1) << 31), "n = %lld out of range", (long long)n);
  REQUIRE(vis_count != nullptr && aligned(vis_count, 8), "vis_count NULL or misaligned");
  if (n == 0) return ok();
  REQUIRE(grad2d != nullptr && vis_idx != nullptr && accum != nullptr && denom != nullptr, "NULL argument");
  REQUIRE(aligned(grad2d, 4) && aligned(vis_idx, 4) && aligned(accum, 4) && aligned(denom, 4), "misaligned array");
  return hip_status(gs::launch_densify_stats(grad2d, vis_idx, vis_count, n, accum, denom,
                                             static_cast<hipStream_t>(stream)),
                    "gs_densify_stats");
}

gs_status gs_densify(const float* params, const float* m, const float* v, int64_t n, int64_t ld,
                     const float* accum, const int32_t* denom, const float* normals, float grad_threshold,
                     float log_scale_threshold, float logit_threshold, float log_shrink, float* out_params,
                     float* out_m, float* out_v, int64_t ld_out, int64_t* out_n, void* workspace,
                     size_t workspace_bytes, void* stream) {
  REQUIRE(n >= 0 && n < (int64_t(1) << 30), "n = %lld out of range", (long long)n);
  REQUIRE(ld >= n && ld >= 1, "ld < n");
  REQUIRE(ld_out >= 0 && ld_out < (int64_t(1) << 31), "ld_out out of range");
  REQUIRE(out_n != nullptr && aligned(out_n, 8), "out_n NULL or misaligned");
  if (n > 0)
    REQUIRE(params && m && v && accum && denom && normals, "NULL params / m / v / accum / denom / normals");
  if (ld_out > 0) REQUIRE(out_params && out_m && out_v, "NULL out_params / out_m / out_v");
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= gs::densify_ws_bytes(n), "workspace too small");
  return hip_status(gs::launch_densify(params, m, v, n, ld, accum, denom, normals, grad_threshold,
                                       log_scale_threshold, logit_threshold, log_shrink, out_params, out_m, out_v,
                                       ld_out, out_n, workspace, static_cast<hipStream_t>(stream)),
                    "gs_densify");
}

gs_status gs_layer_norm_fwd(const void* x, int64_t ldx, const float* gamma, const float* beta, int64_t rows,
                            int32_t width, float eps, int32_t type, void* y, int64_t ldy, float* mean, float* rstd,
                            void* stream) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(width >= 1 && width <= GS_MAX_NET_DIM, "width = %d out of range", int(width));
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps negative or not finite");
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("x", x, ldx, width, elem));
  CHECK(check_matrix("y", y, ldy, width, elem));
  CHECK(check_vector("gamma", gamma));
  CHECK(check_vector("beta", beta));
  CHECK(check_vector("mean", mean));
  CHECK(check_vector("rstd", rstd));
  gs::NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.gamma = gamma;
  a.beta = beta;
  a.rows = int32_t(rows);
  a.width = width;
  a.eps = eps;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  return hip_status(gs::launch_layer_norm_fwd(type, a, static_cast<hipStream_t>(stream)), "gs_layer_norm_fwd");
}

gs_status gs_layer_norm_bwd(const void* x, int64_t ldx, const void* dy, int64_t lddy, const float* gamma,
                            const float* mean, const float* rstd, const void* dres, int64_t lddres, int64_t rows,
                            int32_t width, int32_t type, void* dx, int64_t lddx, float* dgamma, float* dbeta,
                            void* workspace, size_t workspace_bytes, void* stream) {
  CHECK(check_net_sizes(rows, type));
  REQUIRE(width >= 1 && width <= GS_MAX_NET_DIM, "width = %d out of range", int(width));
  const size_t elem = gs::type_bytes(type);
  if (rows > 0) {
    CHECK(check_matrix("x", x, ldx, width, elem));
    CHECK(check_matrix("dy", dy, lddy, width, elem));
    REQUIRE(mean != nullptr && rstd != nullptr, "mean / rstd NULL");
    CHECK(check_vector("mean", mean));
    CHECK(check_vector("rstd", rstd));
    CHECK(check_vector("gamma", gamma));
    if (dres != nullptr) CHECK(check_matrix("dres", dres, lddres, width, elem));
    if (dx != nullptr) CHECK(check_matrix("dx", dx, lddx, width, elem));
  }
  CHECK(check_vector("dgamma", dgamma));
  CHECK(check_vector("dbeta", dbeta));
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  const size_t need = gs::layer_norm_ws_bytes(rows, width);
  REQUIRE(workspace_bytes >= need, "workspace_bytes = %zu < %zu needed", workspace_bytes, need);
  gs::NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.dy = dy;
  a.lddy = lddy;
  a.dres = dres;
  a.lddres = lddres;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.rows = int32_t(rows);
  a.width = width;
  a.dx = dx;
  a.lddx = lddx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  return hip_status(gs::launch_layer_norm_bwd(type, a, workspace, static_cast<hipStream_t>(stream)),
                    "gs_layer_norm_bwd");
}

gs_status gs_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const float* bias,
                        const void* residual, int64_t ldr, int64_t rows, int32_t in, int32_t out, int32_t type,
                        int32_t act, void* y, int64_t ldy, void* z, int64_t ldz, void* stream) {
  gs::LinearArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.bias = bias;
  a.residual = residual;
  a.ldr = ldr;
  a.in = in;
  a.out = out;
  a.act = act;
  a.y = y;
  a.ldy = ldy;
  a.z = z;
  a.ldz = ldz;
  return linear_fwd(a, rows, type, stream, "gs_linear_fwd");
}

gs_status gs_linear_workspace_size(int64_t rows, int32_t in, int32_t out, int32_t num_groups, int32_t type,
                                   int32_t act, size_t* bytes) {
  REQUIRE(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  gs::LinearArgs a{};
  a.in = in;
  a.out = out;
  a.act = act;
  CHECK(check_linear(a, rows, type));
  REQUIRE(num_groups >= 0 && num_groups <= GS_MAX_NET_GROUPS, "num_groups = %d out of range", int(num_groups));
  REQUIRE(gs::linear_fits(rows, in, out, num_groups), "sizes pass a launch grid");
  *bytes = std::max<size_t>(256, gs::linear_bwd_ws_bytes(type, rows, in, out, num_groups, act));
  return ok();
}

gs_status gs_linear_bwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* z, int64_t ldz,
                        const void* dy, int64_t lddy, int64_t rows, int32_t in, int32_t out, int32_t type,
                        int32_t act, void* dx, int64_t lddx, void* dw, int32_t dw_type, float* db, void* workspace,
                        size_t workspace_bytes, void* stream) {
  gs::LinearArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.z = const_cast<void*>(z);
  a.ldz = ldz;
  a.dy = dy;
  a.lddy = lddy;
  a.in = in;
  a.out = out;
  a.act = act;
  a.dx = dx;
  a.lddx = lddx;
  a.dw = dw;
  a.db = db;
  return linear_bwd(a, rows, type, dw_type, workspace, workspace_bytes, stream, "gs_linear_bwd");
}

gs_status gs_grouped_linear_fwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const float* bias,
                                const int64_t* offsets, int32_t num_groups, const void* residual, int64_t ldr,
                                int64_t rows, int32_t in, int32_t out, int32_t type, int32_t act, void* y,
                                int64_t ldy, void* z, int64_t ldz, void* stream) {
  REQUIRE(num_groups >= 1, "num_groups = %d out of range", int(num_groups));
  gs::LinearArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.bias = bias;
  a.offsets = offsets;
  a.groups = num_groups;
  a.residual = residual;
  a.ldr = ldr;
  a.in = in;
  a.out = out;
  a.act = act;
  a.y = y;
  a.ldy = ldy;
  a.z = z;
  a.ldz = ldz;
  return linear_fwd(a, rows, type, stream, "gs_grouped_linear_fwd");
}

gs_status gs_grouped_linear_bwd(const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* offsets,
                                int32_t num_groups, const void* z, int64_t ldz, const void* dy, int64_t lddy,
                                int64_t rows, int32_t in, int32_t out, int32_t type, int32_t act, void* dx,
                                int64_t lddx, void* dw, int32_t dw_type, float* db, void* workspace,
                                size_t workspace_bytes, void* stream) {
  REQUIRE(num_groups >= 1, "num_groups = %d out of range", int(num_groups));
  gs::LinearArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.ldw = ldw;
  a.offsets = offsets;
  a.groups = num_groups;
  a.z = const_cast<void*>(z);
  a.ldz = ldz;
  a.dy = dy;
  a.lddy = lddy;
  a.in = in;
  a.out = out;
  a.act = act;
  a.dx = dx;
  a.lddx = lddx;
  a.dw = dw;
  a.db = db;
  return linear_bwd(a, rows, type, dw_type, workspace, workspace_bytes, stream, "gs_grouped_linear_bwd");
}

gs_status gs_group_sort_workspace_size(int64_t n, int64_t num_groups, size_t* bytes) {
  REQUIRE(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  CHECK(check_sort_sizes(n, num_groups));
  *bytes = gs::group_sort_ws_bytes(n, num_groups);
  return ok();
}

gs_status gs_group_sort(const void* ids, int32_t id_bytes, int64_t n, int64_t num_groups, int64_t* offsets,
                        int32_t* order, int32_t* place, void* workspace, size_t workspace_bytes, void* stream) {
  CHECK(check_sort_sizes(n, num_groups));
  CHECK(check_ids(ids, id_bytes, n));
  REQUIRE(offsets != nullptr && aligned(offsets, 8), "offsets NULL or not 8-byte aligned");
  CHECK(check_vector("order", order));
  CHECK(check_vector("place", place));
  const size_t need = gs::group_sort_ws_bytes(n, num_groups);
  REQUIRE((workspace != nullptr || need == 0) && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  REQUIRE(workspace_bytes >= need, "workspace_bytes = %zu < %zu needed", workspace_bytes, need);
  const gs::SortArgs a{ids, id_bytes, n, num_groups, offsets, order, place};
  return hip_status(gs::launch_group_sort(a, workspace, static_cast<hipStream_t>(stream)), "gs_group_sort");
}

gs_status gs_embedding_fwd(const void* table, int64_t ldt, int64_t num_rows, const void* ids, int32_t id_bytes,
                           int64_t rows, int32_t width, float scale, int32_t type, void* y, int64_t ldy,
                           void* stream) {
  CHECK(check_embedding(rows, num_rows, width, type));
  REQUIRE(std::isfinite(scale), "scale not finite");
  CHECK(check_ids(ids, id_bytes, rows));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("table", table, ldt, width, elem));
  CHECK(check_matrix("y", y, ldy, width, elem));
  gs::EmbedArgs a{};
  a.table = table;
  a.ldt = ldt;
  a.num_rows = num_rows;
  a.ids = ids;
  a.id_bytes = id_bytes;
  a.rows = rows;
  a.width = width;
  a.scale = scale;
  a.y = y;
  a.ldy = ldy;
  return hip_status(gs::launch_embedding_fwd(type, a, static_cast<hipStream_t>(stream)), "gs_embedding_fwd");
}

gs_status gs_embedding_workspace_size(int64_t rows, int64_t num_rows, int32_t width, int32_t type, size_t* bytes) {
  REQUIRE(bytes != nullptr, "bytes is NULL");
  *bytes = 0;
  CHECK(check_embedding(rows, num_rows, width, type));
  *bytes = std::max<size_t>(256, gs::embedding_bwd_ws_bytes(type, rows, num_rows, width));
  return ok();
}

gs_status gs_embedding_bwd(const void* dy, int64_t lddy, const void* ids, int32_t id_bytes, const int64_t* offsets,
                           const int32_t* order, int64_t rows, int64_t num_rows, int32_t width, float scale,
                           int32_t type, void* dtable, int64_t lddt, int32_t dtable_type, void* workspace,
                           size_t workspace_bytes, void* stream) {
  CHECK(check_embedding(rows, num_rows, width, type));
  REQUIRE(std::isfinite(scale), "scale not finite");
  CHECK(check_ids(ids, id_bytes, rows));
  REQUIRE(offsets != nullptr && aligned(offsets, 8), "offsets NULL or not 8-byte aligned");
  if (rows > 0) {
    CHECK(check_matrix("dy", dy, lddy, width, gs::type_bytes(type)));
    REQUIRE(order != nullptr && aligned(order, 4), "order NULL or not 4-byte aligned");
  }
  REQUIRE(dtable_type == type || dtable_type == GS_TYPE_F32, "dtable_type = %d is neither type nor GS_TYPE_F32",
          int(dtable_type));
  CHECK(check_matrix("dtable", dtable, lddt, width, gs::type_bytes(dtable_type)));
  REQUIRE(workspace != nullptr && aligned(workspace, 256), "workspace NULL or not 256-byte aligned");
  const size_t need = gs::embedding_bwd_ws_bytes(type, rows, num_rows, width);
  REQUIRE(workspace_bytes >= need, "workspace_bytes = %zu < %zu needed", workspace_bytes, need);
  gs::EmbedArgs a{};
  a.dy = dy;
  a.lddy = lddy;
  a.ids = ids;
  a.id_bytes = id_bytes;
  a.offsets = offsets;
  a.order = order;
  a.rows = rows;
  a.num_rows = num_rows;
  a.width = width;
  a.scale = scale;
  a.dtable = dtable;
  a.lddt = lddt;
  a.dtable_f32 = dtable_type == GS_TYPE_F32;
  return hip_status(gs::launch_embedding_bwd(type, a, workspace, static_cast<hipStream_t>(stream)),
                    "gs_embedding_bwd");
}

gs_status gs_gate_fwd(const void* logits, int64_t ld, int64_t rows, int32_t groups, int32_t k, int32_t renorm,
                      int32_t type, int32_t* ids, float* weights, void* stream) {
  gs::GateArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.rows = int32_t(rows);
  a.groups = groups;
  a.k = k;
  a.renorm = renorm;
  a.ids = ids;
  a.weights = weights;
  CHECK(check_gate(a, rows, type));
  if (rows == 0) return ok();
  CHECK(check_matrix("logits", logits, ld, groups, gs::type_bytes(type)));
  return hip_status(gs::launch_gate_fwd(type, a, static_cast<hipStream_t>(stream)), "gs_gate_fwd");
}

gs_status gs_gate_bwd(const void* logits, int64_t ld, const int32_t* ids, const float* weights,
                      const float* dweights, int64_t rows, int32_t groups, int32_t k, int32_t renorm, int32_t type,
                      void* dlogits, int64_t lddl, void* stream) {
  gs::GateArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.rows = int32_t(rows);
  a.groups = groups;
  a.k = k;
  a.renorm = renorm;
  a.ids = const_cast<int32_t*>(ids);
  a.weights = const_cast<float*>(weights);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.lddl = lddl;
  CHECK(check_gate(a, rows, type));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("logits", logits, ld, groups, elem));
  CHECK(check_matrix("dlogits", dlogits, lddl, groups, elem));
  REQUIRE(dweights != nullptr && aligned(dweights, 4), "dweights NULL or not 4-byte aligned");
  return hip_status(gs::launch_gate_bwd(type, a, static_cast<hipStream_t>(stream)), "gs_gate_bwd");
}

gs_status gs_dispatch_fwd(const void* x, int64_t ldx, const int32_t* place, int64_t rows, int32_t k, int32_t width,
                          int32_t type, void* xs, int64_t ldxs, void* stream) {
  gs::RouteArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.place = place;
  a.rows = int32_t(rows);
  a.k = k;
  a.width = width;
  a.y = xs;
  a.ldy = ldxs;
  CHECK(check_route(a, rows, type));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("x", x, ldx, width, elem));
  CHECK(check_matrix("xs", xs, ldxs, width, elem));
  return hip_status(gs::launch_dispatch(type, a, static_cast<hipStream_t>(stream)), "gs_dispatch_fwd");
}

gs_status gs_dispatch_bwd(const void* dxs, int64_t lddxs, const int32_t* place, int64_t rows, int32_t k,
                          int32_t width, int32_t type, const void* dres, int64_t ldr, void* dx, int64_t lddx,
                          void* stream) {
  gs::RouteArgs a{};
  a.x = dxs;
  a.ldx = lddxs;
  a.place = place;
  a.rows = int32_t(rows);
  a.k = k;
  a.width = width;
  a.residual = dres;
  a.ldr = ldr;
  a.y = dx;
  a.ldy = lddx;
  CHECK(check_route(a, rows, type));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("dxs", dxs, lddxs, width, elem));
  CHECK(check_matrix("dx", dx, lddx, width, elem));
  return hip_status(gs::launch_combine(type, a, static_cast<hipStream_t>(stream)), "gs_dispatch_bwd");
}

gs_status gs_combine_fwd(const void* ys, int64_t ldys, const int32_t* place, const float* weights,
                         const void* residual, int64_t ldr, int64_t rows, int32_t k, int32_t width, int32_t type,
                         void* y, int64_t ldy, void* stream) {
  gs::RouteArgs a{};
  a.x = ys;
  a.ldx = ldys;
  a.place = place;
  a.weights = weights;
  a.rows = int32_t(rows);
  a.k = k;
  a.width = width;
  a.residual = residual;
  a.ldr = ldr;
  a.y = y;
  a.ldy = ldy;
  CHECK(check_route(a, rows, type));
  if (rows == 0) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("ys", ys, ldys, width, elem));
  CHECK(check_matrix("y", y, ldy, width, elem));
  return hip_status(gs::launch_combine(type, a, static_cast<hipStream_t>(stream)), "gs_combine_fwd");
}

gs_status gs_combine_bwd(const void* dy, int64_t lddy, const void* ys, int64_t ldys, const int32_t* place,
                         const float* weights, int64_t rows, int32_t k, int32_t width, int32_t type, void* dys,
                         int64_t lddys, float* dweights, void* stream) {
  gs::RouteArgs a{};
  a.x = ys;
  a.ldx = ldys;
  a.dy = dy;
  a.lddy = lddy;
  a.place = place;
  a.weights = weights;
  a.rows = int32_t(rows);
  a.k = k;
  a.width = width;
  a.y = dys;
  a.ldy = lddys;
  a.dweights = dweights;
  CHECK(check_route(a, rows, type));
  if (rows == 0 || (dys == nullptr && dweights == nullptr)) return ok();
  const size_t elem = gs::type_bytes(type);
  CHECK(check_matrix("dy", dy, lddy, width, elem));
  if (dweights != nullptr) CHECK(check_matrix("ys", ys, ldys, width, elem));
  if (dys != nullptr) CHECK(check_matrix("dys", dys, lddys, width, elem));
  CHECK(check_vector("dweights", dweights));
  return hip_status(gs::launch_combine_bwd(type, a, static_cast<hipStream_t>(stream)), "gs_combine_bwd");
}

gs_status gs_adamw(const gs_adamw_tensor* tensors, int32_t count, double lr, double beta1, double beta2, double eps,
                   double weight_decay, int64_t step, const int64_t* step_dev, const float* grad_scale,
                   uint64_t seed, void* stream) {
  REQUIRE(count >= 0 && (count == 0 || tensors != nullptr), "count = %d, or tensors NULL", int(count));
  REQUIRE(std::isfinite(lr) && std::isfinite(weight_decay), "lr or weight_decay not finite");
  REQUIRE(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0, "a beta outside [0, 1)");
  // the update's fp32 factors; the hardware's reciprocal takes subnormal numbers as 0
  REQUIRE(float(eps) >= 0x1p-126f && float(eps) <= 0x1p125f, "eps = %g outside [2^-126, 2^125]", eps);
  REQUIRE(std::isfinite(float(lr / (1.0 - beta1))), "lr = %g: too large for fp32 over 1 - beta1", lr);
  REQUIRE(std::isfinite(float(1.0 - lr * weight_decay)), "lr weight_decay = %g too large for fp32", lr * weight_decay);
  REQUIRE(step_dev != nullptr || step >= 1, "step = %lld: 1 or more expected", (long long)step);
  REQUIRE(aligned(step_dev, 8) && aligned(grad_scale, 4), "step_dev or grad_scale misaligned");
  // written ranges, as (first byte, one past the last), sorted to find overlaps
  constexpr int kFew = 64, kRanges = 6;      // tensors; param, m, v, both scales, copy
  std::pair<uintptr_t, uintptr_t> few[kFew * kRanges];
  std::unique_ptr<std::pair<uintptr_t, uintptr_t>[]> more;
  std::pair<uintptr_t, uintptr_t>* ranges = few;
  if (count > kFew) {
    more.reset(new (std::nothrow) std::pair<uintptr_t, uintptr_t>[size_t(count) * kRanges]);
    if (more == nullptr) return fail(GS_ERR_INVALID_ARG, "no host memory for %d tensors", int(count));
    ranges = more.get();
  }
  size_t written = 0;
  auto writes = [&](const void* p, int64_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    ranges[written++] = {at, at + uintptr_t(bytes)};
  };
  bool any[2][3] = {};      // moments in 8 bits, type of the gradients
  for (int32_t i = 0; i < count; ++i) {
    const gs_adamw_tensor& t = tensors[i];
    REQUIRE(t.n >= 0 && t.n <= GS_MAX_ADAMW_SIZE, "tensor %d: n = %lld out of range", int(i), (long long)t.n);
    if (t.n == 0) continue;
    REQUIRE(t.grad_type >= GS_TYPE_BF16 && t.grad_type <= GS_TYPE_F32, "tensor %d: grad_type = %d unknown", int(i),
            int(t.grad_type));
    REQUIRE(t.param != nullptr && aligned(t.param, 4), "tensor %d: param NULL or misaligned", int(i));
    REQUIRE(t.grad != nullptr && aligned(t.grad, gs::type_bytes(t.grad_type)), "tensor %d: grad NULL or misaligned",
            int(i));
    REQUIRE((t.m_scale == nullptr) == (t.v_scale == nullptr), "tensor %d: one scale of two", int(i));
    const bool eight = t.m_scale != nullptr;
    const size_t align = eight ? 1 : 4;
    REQUIRE(t.m != nullptr && t.v != nullptr && aligned(t.m, align) && aligned(t.v, align),
            "tensor %d: m or v NULL or misaligned", int(i));
    REQUIRE(aligned(t.m_scale, 4) && aligned(t.v_scale, 4), "tensor %d: scale misaligned", int(i));
    if (t.copy != nullptr) {
      REQUIRE(t.copy_type >= GS_TYPE_BF16 && t.copy_type <= GS_TYPE_F32, "tensor %d: copy_type = %d unknown", int(i),
              int(t.copy_type));
      REQUIRE(aligned(t.copy, gs::type_bytes(t.copy_type)), "tensor %d: copy misaligned", int(i));
      writes(t.copy, t.n * int64_t(gs::type_bytes(t.copy_type)));
    }
    writes(t.param, t.n * 4);
    writes(t.m, t.n * (eight ? 1 : 4));
    writes(t.v, t.n * (eight ? 1 : 4));
    if (eight) {
      const int64_t blocks = (t.n + GS_ADAMW_BLOCK - 1) / GS_ADAMW_BLOCK;
      writes(t.m_scale, blocks * 4);
      writes(t.v_scale, blocks * 4);
    }
    any[eight][t.grad_type] = true;
  }
  std::sort(ranges, ranges + written);
  for (size_t i = 1; i < written; ++i) REQUIRE(ranges[i].first >= ranges[i - 1].second, "written ranges overlap");
  const gs::AdamwHyper h{lr, beta1, beta2, eps, weight_decay, step, step_dev, grad_scale};
  for (int kind = 0; kind < 6; ++kind) {
    const bool eight = kind >= 3;
    const int type = kind % 3;
    if (!any[eight][type]) continue;
    gs::AdamwTensor batch[gs::kAdamwTensors];
    int held = 0;
    uint32_t workgroups = 0;
    for (int32_t i = 0; i <= count; ++i) {
      const bool take = i < count && tensors[i].n > 0 && (tensors[i].m_scale != nullptr) == eight &&
                        tensors[i].grad_type == type;
      const uint32_t mine = take ? gs::adamw_workgroups(tensors[i].n) : 0;
      // a launch ends with its room for tensors, or where its threads would pass 2^32 - 1
      if (held > 0 && (i == count || (take && (held == gs::kAdamwTensors || workgroups + mine >= (1u << 24))))) {
        const hipError_t e =
            gs::launch_adamw(batch, held, eight, type, workgroups, h, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_status(e, "gs_adamw");
        held = 0;
        workgroups = 0;
      }
      if (!take) continue;
      const gs_adamw_tensor& t = tensors[i];
      batch[held++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n, workgroups,
                       gs::adamw_key(seed, uint32_t(i)), t.copy_type};
      workgroups += mine;
    }
  }
  return ok();
}

gs_status gs_adamw_moment(const uint8_t* codes, const float* scales, int64_t n, int32_t moment, int32_t type,
                          void* values, void* stream) {
  REQUIRE(n >= 0 && n <= GS_MAX_ADAMW_SIZE, "n = %lld out of range", (long long)n);
  REQUIRE(moment == 1 || moment == 2, "moment = %d: 1 or 2 expected", int(moment));
  REQUIRE(type >= GS_TYPE_BF16 && type <= GS_TYPE_F32, "type = %d unknown", int(type));
  if (n == 0) return ok();
  REQUIRE(codes != nullptr, "codes is NULL");
  REQUIRE(scales != nullptr && aligned(scales, 4), "scales NULL or misaligned");
  REQUIRE(values != nullptr && aligned(values, gs::type_bytes(type)), "values NULL or misaligned");
  return hip_status(gs::launch_adamw_moment(codes, scales, n, moment, type, values, static_cast<hipStream_t>(stream)),
                    "gs_adamw_moment");
}

}  // extern "C"
