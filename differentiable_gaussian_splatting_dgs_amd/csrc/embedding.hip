// Rows looked up in a table, and the table's gradient by sorted ids.
//
//   forward   y[i] = scale table[id[i]], zeros for an id outside the table
//   backward  dtable[v] = scale sum of dy[i] over id[i] = v
//
// Both are bound by the bytes of the rows.  Sums are fp32; the rounding into
// the storage type is the last step.
#include <algorithm>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t id_at(const void* __restrict__ ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// L lanes a row.
template <typename T, int L>
__global__ __launch_bounds__(kThreads) void k_lookup(EmbedArgs a) {
  constexpr int K = kChunk<T>;
  const Row<T> row(a.width);
  constexpr int kRows = kThreads / L;
  for (int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / L; r < a.rows; r += int64_t(gridDim.x) * kRows) {
    const int64_t id = id_at(a.ids, a.id_bytes, r);
    const bool there = id >= 0 && id < a.num_rows;
    const T* __restrict__ src = static_cast<const T*>(a.table) + (there ? id : 0) * a.ldt;
    T* __restrict__ dst = static_cast<T*>(a.y) + r * a.ldy;
    for (int c = threadIdx.x % L; c < row.chunks; c += L) {
      float v[K] = {};
      if (there) {
        const Chunk<T> x = row.load(src, c);
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = float(x.v[i]) * a.scale;
      }
      row.store(dst, c, v);
    }
  }
}

// L lanes a row of the table.
template <typename T, typename O, int L>
__global__ __launch_bounds__(kThreads) void k_table_grad(EmbedArgs a) {
  constexpr int K = kChunk<T>;
  const Row<T> row(a.width);
  constexpr int kRows = kThreads / L;
  for (int64_t v = int64_t(blockIdx.x) * kRows + threadIdx.x / L; v < a.num_rows; v += int64_t(gridDim.x) * kRows) {
    const int64_t p0 = std::max<int64_t>(a.offsets[v], 0), p1 = std::min<int64_t>(a.offsets[v + 1], a.rows);
    for (int c = threadIdx.x % L; c < row.chunks; c += L) {
      float sum[K] = {};
      for (int64_t p = p0; p < p1; ++p) {
        const int64_t r = a.order[p];
        if (r < 0 || r >= a.rows) continue;
        const Chunk<T> x = row.load(static_cast<const T*>(a.dy) + r * a.lddy, c);
#pragma unroll
        for (int i = 0; i < K; ++i) sum[i] += float(x.v[i]);
      }
#pragma unroll
      for (int i = 0; i < K; ++i) sum[i] *= a.scale;
      row.store(static_cast<O*>(a.dtable) + v * a.lddt, c, sum);
    }
  }
}

template <typename T, int L>
hipError_t go_fwd(const EmbedArgs& a, hipStream_t st) {
  k_lookup<T, L><<<grid_of((a.rows + kThreads / L - 1) / (kThreads / L)), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int L>
hipError_t go_bwd(const EmbedArgs& a, hipStream_t st) {
  const unsigned grid = grid_of((a.num_rows + kThreads / L - 1) / (kThreads / L));
  if (a.dtable_f32)
    k_table_grad<T, float, L><<<grid, kThreads, 0, st>>>(a);
  else
    k_table_grad<T, T, L><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t embed_fwd(const EmbedArgs& a, hipStream_t st) {
  switch (row_lanes((a.width + kChunk<T> - 1) / kChunk<T>)) {
    case 8: return go_fwd<T, 8>(a, st);
    case 16: return go_fwd<T, 16>(a, st);
    case 32: return go_fwd<T, 32>(a, st);
    default: return go_fwd<T, 64>(a, st);
  }
}

template <typename T>
hipError_t embed_bwd(const EmbedArgs& a, hipStream_t st) {
  switch (row_lanes((a.width + kChunk<T> - 1) / kChunk<T>)) {
    case 8: return go_bwd<T, 8>(a, st);
    case 16: return go_bwd<T, 16>(a, st);
    case 32: return go_bwd<T, 32>(a, st);
    default: return go_bwd<T, 64>(a, st);
  }
}

}  // namespace
}  // namespace net

size_t embedding_bwd_ws_bytes(int, int64_t, int64_t, int32_t) { return 256; }

hipError_t launch_embedding_fwd(int type, const EmbedArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return net::embed_fwd<net::bf16>(a, st);
  if (type == kTypeF16) return net::embed_fwd<net::f16>(a, st);
  return net::embed_fwd<float>(a, st);
}

hipError_t launch_embedding_bwd(int type, const EmbedArgs& a, void*, hipStream_t st) {
  if (type == kTypeBF16) return net::embed_bwd<net::bf16>(a, st);
  if (type == kTypeF16) return net::embed_bwd<net::f16>(a, st);
  return net::embed_bwd<float>(a, st);
}

}  // namespace gs
