// Rows to the places that the sort by group gave their choices, and back with
// weights, each with its gradient.
//
//   dispatch       xs[place[i][j]] = x[i]
//   combine        y[i] = sum_j w[i][j] ys[place[i][j]] + residual[i]
//                  (w = 1: dispatch's gradient, residual the gradient past it)
//   combine's gradient   dys[place[i][j]] = w[i][j] dy[i],
//                  dw[i][j] = sum over the columns of dy[i] ys[place[i][j]]
//
// All go by the row i, not by the sorted position: x and dy are read once
// for all k choices, the sums over j need no atomics and have a fixed order.
// Bound by the bytes of the rows.  Sums are fp32; the rounding into storage is
// the last step.  400,000 x 256 bf16 to two places each: 98 to 102 us (614 MB at
// 6.1 TB/s, two thirds of it writes); 131,072 x 1024 fp16 from four places with the
// residual: 282 us (1.61 GB at 5.7 TB/s); gradients of 65,537 x 515 fp32, two
// places: 130 us (677 MB at 5.2 TB/s; with one chunk of a lane in flight 148).
#include <algorithm>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;

// The row's places, -1 for one outside its range.
template <int KM>
__device__ __forceinline__ void load_places(const RouteArgs& a, int64_t r, int32_t (&at)[KM]) {
  const int32_t most = a.rows * a.k;
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    at[j] = j < a.k ? a.place[r * a.k + j] : -1;
    if (uint32_t(at[j]) >= uint32_t(most)) at[j] = -1;
  }
}

template <int KM>
__device__ __forceinline__ void load_weights(const RouteArgs& a, int64_t r, float (&w)[KM]) {
#pragma unroll
  for (int j = 0; j < KM; ++j) w[j] = a.weights != nullptr && j < a.k ? a.weights[r * a.k + j] : 1.0f;
}

// Items are slices of rows: L lanes, a chunk for each.
template <int L>
__device__ __forceinline__ int64_t first_item() {
  return int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
}
template <int L>
__device__ __forceinline__ int64_t next_item() {
  return int64_t(gridDim.x) * (kThreads / L);
}

template <typename T, int L, int KM, bool kFar, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_dispatch(RouteArgs a, int slices) {
  const Row<T, kNarrow> row(a.width);
  T* const xs = static_cast<T*>(a.y);
  for (int64_t item = first_item<L>(); item < int64_t(a.rows) * slices; item += next_item<L>()) {
    const int64_t r = item / slices;
    const int c = int(item - r * slices) * L + threadIdx.x % L;
    if (c >= row.chunks) continue;
    const Chunk<T> x = row.load(static_cast<const T*>(a.x) + r * a.ldx, c);
    int32_t at[KM];
    load_places<KM>(a, r, at);
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (at[j] >= 0) row.template copy<kFar>(xs + at[j] * a.ldy, c, x);
  }
}

template <typename T, int L, int KM, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_combine(RouteArgs a, int slices) {
  constexpr int K = kChunk<T>;
  const Row<T, kNarrow> row(a.width);
  const T* const ys = static_cast<const T*>(a.x);
  for (int64_t item = first_item<L>(); item < int64_t(a.rows) * slices; item += next_item<L>()) {
    const int64_t r = item / slices;
    const int c = int(item - r * slices) * L + threadIdx.x % L;
    if (c >= row.chunks) continue;
    int32_t at[KM];
    float w[KM];
    load_places<KM>(a, r, at);
    load_weights<KM>(a, r, w);
    // a place that was left out reads row 0, and drops it
    Chunk<T> v[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) v[j] = row.load(ys + (at[j] < 0 ? 0 : at[j]) * a.ldx, c);
    float sum[K] = {};
#pragma unroll
    for (int j = 0; j < KM; ++j)
#pragma unroll
      for (int i = 0; i < K; ++i) sum[i] = at[j] < 0 ? sum[i] : fmaf(w[j], float(v[j].v[i]), sum[i]);
    T* const y = static_cast<T*>(a.y) + r * a.ldy;
    if (a.residual != nullptr) {
      const Chunk<T> res = row.load(static_cast<const T*>(a.residual) + r * a.ldr, c);
#pragma unroll
      for (int i = 0; i < K; ++i) sum[i] += float(res.v[i]);
    }
    if (a.residual == a.y)
      row.store_rest(y, c, sum);
    else
      row.store(y, c, sum);
  }
}

// L lanes a row, which they walk C chunks a lane at a time: the products' sums
// stay in registers.
template <typename T, int L, int C, int KM, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_combine_bwd(RouteArgs a) {
  constexpr int K = kChunk<T>;
  const Row<T, kNarrow> row(a.width);
  const int l = threadIdx.x % L;
  const T* const ys = static_cast<const T*>(a.x);
  T* const dys = static_cast<T*>(a.y);
  // all lanes of a row together
  for (int64_t r = first_item<L>(); r < a.rows; r += next_item<L>()) {
    int32_t at[KM];
    float w[KM], dot[KM] = {};
    load_places<KM>(a, r, at);
    load_weights<KM>(a, r, w);
    const T* const dy = static_cast<const T*>(a.dy) + r * a.lddy;
    for (int c0 = l; c0 < row.chunks; c0 += L * C) {
      int c[C];      // past the row's end: its last chunk, which does not count
      Chunk<T> g[C];
#pragma unroll
      for (int q = 0; q < C; ++q) {
        c[q] = std::min(c0 + q * L, row.chunks - 1);
        g[q] = row.load(dy, c[q]);
      }
      if (a.dweights != nullptr) {
        Chunk<T> v[C][KM];
#pragma unroll
        for (int q = 0; q < C; ++q)
#pragma unroll
          for (int j = 0; j < KM; ++j) v[q][j] = row.load(ys + (at[j] < 0 ? 0 : at[j]) * a.ldx, c[q]);
#pragma unroll
        for (int q = 0; q < C; ++q) {
          const int skip = c0 + q * L < row.chunks ? row.again(c[q]) : K;
#pragma unroll
          for (int j = 0; j < KM; ++j)
#pragma unroll
            for (int i = 0; i < K; ++i)
              dot[j] = i < skip ? dot[j] : fmaf(float(g[q].v[i]), float(v[q][j].v[i]), dot[j]);
        }
      }
      if (dys != nullptr)
#pragma unroll
        for (int q = 0; q < C; ++q)
#pragma unroll
          for (int j = 0; j < KM; ++j)
            if (at[j] >= 0 && c0 + q * L < row.chunks) {
              float o[K];
#pragma unroll
              for (int i = 0; i < K; ++i) o[i] = w[j] * float(g[q].v[i]);
              row.store(dys + at[j] * a.ldy, c[q], o);
            }
    }
    if (a.dweights == nullptr) continue;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
#pragma unroll
      for (int d = 1; d < L; d <<= 1) dot[j] += __shfl_xor(dot[j], d, 64);
      if (j < a.k && l == 0) a.dweights[r * a.k + j] = at[j] < 0 ? 0.0f : dot[j];
    }
  }
}

enum Way { kDispatch, kCombine, kCombineBwd };

template <typename T, int KM>
hipError_t go_by_chunks(const RouteArgs& a, int64_t chunks, hipStream_t st) {
  k_combine<T, 1, KM, false><<<grid_of((a.rows * chunks + kThreads - 1) / kThreads), kThreads, 0, st>>>(a, int(chunks));
  return hipGetLastError();
}

template <typename T, int L, int KM, bool kNarrow>
hipError_t go(Way way, const RouteArgs& a, hipStream_t st) {
  // rows of several chunks a lane: as many in flight as registers allow
  constexpr int kAhead = L != 64 ? 1 : KM <= 2 ? 3 : KM <= 4 ? 2 : 1;
  const int64_t chunks = (a.width + kChunk<T> - 1) / kChunk<T>;
  // Rows back from one place or two keep few loads in flight, and a wave for the
  // end of a row has idle lanes: such rows by the chunk, wherever a wave begins.
  // 300,000 x 258 fp32 from one place 196 -> 137 us, 150,000 from two 104 -> 91, from
  // four 75 and 73 either way; to their places such rows take longer by the chunk (138 ->
  // 156), since two workgroups then write the same lines.
  if constexpr (L == 64 && KM <= 2)
    if (way == kCombine && chunks % 64 != 0 && chunks > 64) return go_by_chunks<T, KM>(a, chunks, st);
  const int64_t slices = way == kCombineBwd ? 1 : (chunks + L - 1) / L;
  const unsigned grid = grid_of((a.rows * slices + kThreads / L - 1) / (kThreads / L));
  if (way == kDispatch && is_far(a.y, a.ldy, int64_t(a.rows) * a.k, sizeof(T)))
    k_dispatch<T, L, KM, true, kNarrow><<<grid, kThreads, 0, st>>>(a, int(slices));
  else if (way == kDispatch)
    k_dispatch<T, L, KM, false, kNarrow><<<grid, kThreads, 0, st>>>(a, int(slices));
  else if (way == kCombine)
    k_combine<T, L, KM, kNarrow><<<grid, kThreads, 0, st>>>(a, int(slices));
  else if (kAhead > 1 && a.width > 64 * kChunk<T>)
    k_combine_bwd<T, L, kAhead, KM, kNarrow><<<grid, kThreads, 0, st>>>(a);
  else
    k_combine_bwd<T, L, 1, KM, kNarrow><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int L, bool kNarrow = false>
hipError_t by_choices(Way way, const RouteArgs& a, hipStream_t st) {
  if (a.k <= 1) return go<T, L, 1, kNarrow>(way, a, st);
  if (a.k <= 2) return go<T, L, 2, kNarrow>(way, a, st);
  if (a.k <= 4) return go<T, L, 4, kNarrow>(way, a, st);
  if (a.k <= 8) return go<T, L, 8, kNarrow>(way, a, st);
  return go<T, L, kMaxChoices, kNarrow>(way, a, st);
}

template <typename T>
hipError_t by_width(Way way, const RouteArgs& a, hipStream_t st) {
  if (a.width < kChunk<T>) return by_choices<T, 8, true>(way, a, st);
  switch (row_lanes((a.width + kChunk<T> - 1) / kChunk<T>)) {
    case 8: return by_choices<T, 8>(way, a, st);
    case 16: return by_choices<T, 16>(way, a, st);
    case 32: return by_choices<T, 32>(way, a, st);
    default: return by_choices<T, 64>(way, a, st);
  }
}

hipError_t by_type(int type, Way way, const RouteArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return by_width<bf16>(way, a, st);
  if (type == kTypeF16) return by_width<f16>(way, a, st);
  return by_width<float>(way, a, st);
}

}  // namespace
}  // namespace net

hipError_t launch_dispatch(int type, const RouteArgs& a, hipStream_t st) {
  return net::by_type(type, net::kDispatch, a, st);
}
hipError_t launch_combine(int type, const RouteArgs& a, hipStream_t st) {
  return net::by_type(type, net::kCombine, a, st);
}
hipError_t launch_combine_bwd(int type, const RouteArgs& a, hipStream_t st) {
  return net::by_type(type, net::kCombineBwd, a, st);
}

}  // namespace gs
