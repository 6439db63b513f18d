// The linear layer's dispatch by storage type, and what its grids can hold.
#include <algorithm>

#include "gs_internal.h"

namespace gs {

hipError_t linear_fwd_bf16(const LinearArgs& a, hipStream_t st);
hipError_t linear_fwd_f16(const LinearArgs& a, hipStream_t st);
hipError_t linear_fwd_f32(const LinearArgs& a, hipStream_t st);
hipError_t linear_bwd_bf16(const LinearArgs& a, char* ws, hipStream_t st);
hipError_t linear_bwd_f16(const LinearArgs& a, char* ws, hipStream_t st);
hipError_t linear_bwd_f32(const LinearArgs& a, char* ws, hipStream_t st);
size_t linear_bwd_ws_bf16(int64_t rows, int32_t in, int32_t out, int32_t groups, int act);
size_t linear_bwd_ws_f16(int64_t rows, int32_t in, int32_t out, int32_t groups, int act);
size_t linear_bwd_ws_f32(int64_t rows, int32_t in, int32_t out, int32_t groups, int act);

bool linear_fits(int64_t rows, int32_t in, int32_t out, int32_t groups) {
  // 256 threads a workgroup and a launch below 2^32 threads, which dx's and
  // dw's tiles may share; the smallest tile is 64 x 64
  const int64_t most = int64_t(1) << 23, side = std::max(in, out);
  const int64_t high = rows / 64 + std::max(groups, 1), wide = (side + 63) / 64;
  const int64_t planes = ((int64_t(in) + 63) / 64) * ((int64_t(out) + 63) / 64);
  return high * wide < most && (planes + 768) * (std::max(groups, 1) + 1) < most;
}

size_t linear_bwd_ws_bytes(int type, int64_t rows, int32_t in, int32_t out, int32_t groups, int act) {
  if (type == kTypeBF16) return linear_bwd_ws_bf16(rows, in, out, groups, act);
  if (type == kTypeF16) return linear_bwd_ws_f16(rows, in, out, groups, act);
  return linear_bwd_ws_f32(rows, in, out, groups, act);
}

hipError_t launch_linear_fwd(int type, const LinearArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (type == kTypeBF16) return linear_fwd_bf16(a, st);
  if (type == kTypeF16) return linear_fwd_f16(a, st);
  return linear_fwd_f32(a, st);
}

hipError_t launch_linear_bwd(int type, const LinearArgs& a, void* ws, hipStream_t st) {
  if (type == kTypeBF16) return linear_bwd_bf16(a, static_cast<char*>(ws), st);
  if (type == kTypeF16) return linear_bwd_f16(a, static_cast<char*>(ws), st);
  return linear_bwd_f32(a, static_cast<char*>(ws), st);
}

}  // namespace gs
