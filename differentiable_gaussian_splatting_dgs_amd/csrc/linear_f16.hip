// The linear layer for f16 storage (linear_kernels.hpp).
#include "linear_kernels.hpp"

namespace gs {

hipError_t linear_fwd_f16(const LinearArgs& a, hipStream_t st) { return net::linear_fwd<net::f16>(a, st); }
hipError_t linear_bwd_f16(const LinearArgs& a, char* ws, hipStream_t st) { return net::linear_bwd<net::f16>(a, ws, st); }
size_t linear_bwd_ws_f16(int64_t rows, int32_t in, int32_t out, int32_t groups, int act) {
  return net::bwd_plan<net::f16>(rows, in, out, groups, act).total;
}

}  // namespace gs
