// The linear layer for f32 storage (linear_kernels.hpp).
#include "linear_kernels.hpp"

namespace gs {

hipError_t linear_fwd_f32(const LinearArgs& a, hipStream_t st) { return net::linear_fwd<float>(a, st); }
hipError_t linear_bwd_f32(const LinearArgs& a, char* ws, hipStream_t st) { return net::linear_bwd<float>(a, ws, st); }
size_t linear_bwd_ws_f32(int64_t rows, int32_t in, int32_t out, int32_t groups, int act) {
  return net::bwd_plan<float>(rows, in, out, groups, act).total;
}

}  // namespace gs
