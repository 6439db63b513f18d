// The gate: the k largest logits of a row with their softmax weights, and the
// gradient of the logits.
//
//   forward   k times the largest logit left, ties to the lower index; weights
//             e^(l - m) / sum e^(l - m), m the largest, the sum over the chosen
//             (renorm) or over all
//   backward  renorm: dl = w (dw - s) where chosen, s = sum w dw; else
//             dl = [chosen] w dw - p s, p = w_0 e^(l - l_0), 0 the first choice:
//             the row's maximum and sum are not worked out again
//
// A row lies in the registers of L lanes, read once.  A logit becomes an
// unsigned number that orders as it does, with its column below it, so that a
// maximum of numbers is the choice: 32 bits for 16-bit logits, 64 for fp32.
// Bound by the bytes of the logits.
#include <algorithm>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;

// Orders as x does: NaN above all, -0 as 0; never 0.
__device__ __forceinline__ uint32_t rank_of(float x) {
  x += 0.0f;
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t rank) {
  return __builtin_bit_cast(float, (rank >> 31) != 0 ? rank & 0x7FFFFFFFu : ~rank);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;      // rank_of(-inf)

// The numbers compared: rank, then the lower column.  0: no logit.
template <typename T>
struct Pick {      // fp32
  using U = uint64_t;
  static __device__ __forceinline__ U make(T x, int col) { return U(rank_of(x)) << 32 | (0xFFFFu - col); }
  static __device__ __forceinline__ float value(U u) { return value_of(uint32_t(u >> 32)); }
  static __device__ __forceinline__ bool none(U u) { return uint32_t(u >> 32) <= kMinusInf; }
  static __device__ __forceinline__ int column(U u) { return 0xFFFF - int(uint32_t(u) & 0xFFFFu); }
};

template <typename T>
struct Pick16 {
  using U = uint32_t;
  static __device__ __forceinline__ U make(T x, int col) {
    uint32_t b = __builtin_bit_cast(uint16_t, x);
    const float f = float(x);
    b = f == 0.0f ? 0x8000u : (b >> 15) != 0 ? b ^ 0xFFFFu : b | 0x8000u;
    return (f != f ? 0xFFFFu : b) << 16 | (0xFFFFu - col);
  }
  static __device__ __forceinline__ T stored(U u) {
    const uint32_t b = u >> 16;
    return __builtin_bit_cast(T, uint16_t((b >> 15) != 0 ? b & 0x7FFFu : ~b));
  }
  static __device__ __forceinline__ float value(U u) { return float(stored(u)); }
  static __device__ __forceinline__ bool none(U u) { return u == 0 || value(u) == -__builtin_inff(); }
  static __device__ __forceinline__ int column(U u) { return 0xFFFF - int(u & 0xFFFFu); }
};
template <>
struct Pick<bf16> : Pick16<bf16> {};
template <>
struct Pick<f16> : Pick16<f16> {};

template <typename U>
__device__ __forceinline__ U larger(U a, U b) { return a > b ? a : b; }

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v = larger(v, uint32_t(__shfl_xor(int(v), d, 64)));
  return v;
}
template <int L>
__device__ __forceinline__ uint64_t row_max(uint64_t v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    const uint64_t o = uint64_t(uint32_t(__shfl_xor(int(v >> 32), d, 64))) << 32 |
                       uint32_t(__shfl_xor(int(v), d, 64));
    v = larger(v, o);
  }
  return v;
}

// L lanes a row, C chunks a lane; KM: choices, rounded up.
template <typename T, int L, int C, int KM>
__device__ __forceinline__ void gate_row(const GateArgs& a, int64_t r, int l) {
  constexpr int K = kChunk<T>;
  using P = Pick<T>;
  using U = typename P::U;
  const T* __restrict__ x = static_cast<const T*>(a.logits) + r * a.ld;
  U u[C][K];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c0 = (l + L * j) * K, n = std::min(K, std::max(0, a.groups - c0));
    const Chunk<T> v = load_chunk_n(x + (n > 0 ? c0 : 0), n);
#pragma unroll
    for (int i = 0; i < K; ++i) u[j][i] = i < n ? P::make(v.v[i], c0 + i) : U(0);
  }
  float e[KM];
  int32_t id[KM];
  float top = 0.0f, total = 0.0f;
#pragma unroll
  for (int q = 0; q < KM; ++q) {
    U best = 0;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < K; ++i) best = larger(best, u[j][i]);
    best = row_max<L>(best);
    const bool none = P::none(best);
    if (q == 0) {
      top = none ? 0.0f : P::value(best);
      if (a.renorm == 0) {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < K; ++i) total += P::none(u[j][i]) ? 0.0f : expf(P::value(u[j][i]) - top);
#pragma unroll
        for (int d = 1; d < L; d <<= 1) total += __shfl_xor(total, d, 64);
      }
    }
    id[q] = none ? -1 : P::column(best);
    e[q] = none ? 0.0f : expf(P::value(best) - top);
    if (a.renorm != 0 && q < a.k) total += e[q];
    // columns are distinct, so one element is the choice
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < K; ++i) u[j][i] = u[j][i] == best ? U(0) : u[j][i];
  }
  const bool dead = id[0] < 0;
#pragma unroll
  for (int q = 0; q < KM; ++q)
    if (q < a.k && (q & (L - 1)) == l) {
      a.ids[r * a.k + q] = id[q];
      a.weights[r * a.k + q] = dead || id[q] < 0 ? 0.0f : e[q] / total;
    }
}

template <typename T, int L, int C, int KM>
__device__ __forceinline__ void gate_row_bwd(const GateArgs& a, int64_t r, int l) {
  constexpr int K = kChunk<T>;
  const T* __restrict__ x = static_cast<const T*>(a.logits) + r * a.ld;
  T* __restrict__ dl = static_cast<T*>(a.dlogits) + r * a.lddl;
  int32_t id[KM];
  float part[KM], w[KM], s = 0.0f;
#pragma unroll
  for (int q = 0; q < KM; ++q) {
    id[q] = q < a.k ? a.ids[r * a.k + q] : -1;
    if (uint32_t(id[q]) >= uint32_t(a.groups)) id[q] = -1;
    w[q] = id[q] < 0 ? 0.0f : a.weights[r * a.k + q];
    part[q] = id[q] < 0 ? 0.0f : w[q] * a.dweights[r * a.k + q];
    s += part[q];
  }
  float first = 0.0f;
  if (a.renorm != 0) {
#pragma unroll
    for (int q = 0; q < KM; ++q) part[q] -= w[q] * s;
  } else if (id[0] >= 0) {
    first = float(x[id[0]]);
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c0 = (l + L * j) * K, n = std::min(K, std::max(0, a.groups - c0));
    if (n == 0) continue;
    float g[K] = {};
    if (a.renorm == 0 && id[0] >= 0) {
      const Chunk<T> v = load_chunk_n(x + c0, n);
#pragma unroll
      for (int i = 0; i < K; ++i) g[i] = -(w[0] * expf(float(v.v[i]) - first)) * s;
    }
#pragma unroll
    for (int q = 0; q < KM; ++q)
#pragma unroll
      for (int i = 0; i < K; ++i) g[i] += id[q] == c0 + i ? part[q] : 0.0f;
    Chunk<T> o;
#pragma unroll
    for (int i = 0; i < K; ++i) o.v[i] = T(g[i]);
    store_chunk_n(dl + c0, o, n);
  }
}

template <typename T, int L, int C, int KM, bool kFwd>
__global__ __launch_bounds__(kThreads) void k_gate(GateArgs a) {
  constexpr int kRows = kThreads / L;
  // all lanes of a row together
  for (int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / L; r < a.rows; r += int64_t(gridDim.x) * kRows) {
    if constexpr (kFwd)
      gate_row<T, L, C, KM>(a, r, threadIdx.x % L);
    else
      gate_row_bwd<T, L, C, KM>(a, r, threadIdx.x % L);
  }
}

template <typename T, int L, int C, int KM>
hipError_t go(bool fwd, const GateArgs& a, hipStream_t st) {
  const unsigned grid = grid_of((int64_t(a.rows) + kThreads / L - 1) / (kThreads / L));
  if (fwd)
    k_gate<T, L, C, KM, true><<<grid, kThreads, 0, st>>>(a);
  else
    k_gate<T, L, C, KM, false><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int L, int C>
hipError_t by_choices(bool fwd, const GateArgs& a, hipStream_t st) {
  if (a.k <= 1) return go<T, L, C, 1>(fwd, a, st);
  if (a.k <= 2) return go<T, L, C, 2>(fwd, a, st);
  if (a.k <= 4) return go<T, L, C, 4>(fwd, a, st);
  if (a.k <= 8) return go<T, L, C, 8>(fwd, a, st);
  return go<T, L, C, kMaxChoices>(fwd, a, st);
}

template <typename T>
hipError_t by_width(bool fwd, const GateArgs& a, hipStream_t st) {
  const int chunks = (a.groups + kChunk<T> - 1) / kChunk<T>;
  if (chunks <= 8) return by_choices<T, 8, 1>(fwd, a, st);
  if (chunks <= 16) return by_choices<T, 16, 1>(fwd, a, st);
  if (chunks <= 32) return by_choices<T, 32, 1>(fwd, a, st);
  if (chunks <= 64) return by_choices<T, 64, 1>(fwd, a, st);
  if constexpr (sizeof(T) == 4)
    if (chunks > 128) return by_choices<T, 64, 4>(fwd, a, st);
  return by_choices<T, 64, 2>(fwd, a, st);
}

hipError_t by_type(int type, bool fwd, const GateArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return by_width<bf16>(fwd, a, st);
  if (type == kTypeF16) return by_width<f16>(fwd, a, st);
  return by_width<float>(fwd, a, st);
}

}  // namespace
}  // namespace net

hipError_t launch_gate_fwd(int type, const GateArgs& a, hipStream_t st) { return net::by_type(type, true, a, st); }
hipError_t launch_gate_bwd(int type, const GateArgs& a, hipStream_t st) { return net::by_type(type, false, a, st); }

}  // namespace gs
