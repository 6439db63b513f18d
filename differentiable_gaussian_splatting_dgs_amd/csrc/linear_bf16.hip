// The linear layer for bf16 storage (linear_kernels.hpp).
#include "linear_kernels.hpp"

namespace gs {

hipError_t linear_fwd_bf16(const LinearArgs& a, hipStream_t st) { return net::linear_fwd<net::bf16>(a, st); }
hipError_t linear_bwd_bf16(const LinearArgs& a, char* ws, hipStream_t st) { return net::linear_bwd<net::bf16>(a, ws, st); }
size_t linear_bwd_ws_bf16(int64_t rows, int32_t in, int32_t out, int32_t groups, int act) {
  return net::bwd_plan<net::bf16>(rows, in, out, groups, act).total;
}

}  // namespace gs
