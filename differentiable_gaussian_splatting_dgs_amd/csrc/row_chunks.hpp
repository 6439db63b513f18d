// Rows in 16-byte chunks for the operators that copy, scale and sum whole
// rows (embedding.hip, route.hip).
#pragma once

#include "net_common.hpp"

namespace gs {
namespace net {

// A row of at least one chunk's width is covered by whole chunks, the last
// one moved back onto the row's end, so that no width takes a slower path:
// what two chunks share is read twice and written twice with the same values.
// A narrower row is one part of a chunk.
template <typename T>
struct Row {
  static constexpr int K = kChunk<T>;
  int width, chunks;
  __device__ __forceinline__ explicit Row(int w) : width(w), chunks((w + K - 1) / K) {}
  __device__ __forceinline__ int at(int c) const {     // first column of chunk c
    return width < K ? 0 : (c * K + K <= width ? c * K : width - K);
  }
  __device__ __forceinline__ int again(int c) const {  // its columns that the chunk before has too
    return c * K - at(c);
  }
  __device__ __forceinline__ Chunk<T> load(const T* __restrict__ row, int c) const {
    return width >= K ? load_chunk(row + at(c)) : load_chunk_n(row, width);
  }
  template <typename O>      // O of T's size, or fp32 for 16-bit T
  __device__ __forceinline__ void store(O* __restrict__ row, int c, const float (&v)[K]) const {
    if constexpr (sizeof(O) == sizeof(T)) {
      Chunk<O> o;
#pragma unroll
      for (int i = 0; i < K; ++i) o.v[i] = O(v[i]);
      if (width >= K)
        store_chunk(row + at(c), o);
      else
        store_chunk_n(row, o, width);
    } else {
      if (width >= K) {
#pragma unroll
        for (int h = 0; h < K; h += 4) {
          Chunk<float> o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o.v[i] = v[h + i];
          store_chunk(row + at(c) + h, o);
        }
      } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (i < width) row[i] = v[i];
      }
    }
  }
  __device__ __forceinline__ void copy(T* __restrict__ row, int c, const Chunk<T>& v) const {
    if (width >= K)
      store_chunk(row + at(c), v);
    else
      store_chunk_n(row, v, width);
  }
  // Without the columns that the chunk before has too: what rows that are
  // read and written in place need.
  __device__ __forceinline__ void store_rest(T* __restrict__ row, int c, const float (&v)[K]) const {
    if (width < K || again(c) == 0) {
      store(row, c, v);
      return;
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (i >= again(c)) row[at(c) + i] = T(v[i]);
  }
};

// Lanes that share a row: a power of two, 8 ... 64, that leaves few of them
// without a chunk.
inline int row_lanes(int chunks) { return chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64; }

// A launch takes less than 2^32 threads: kernels whose items may be more walk
// them with the grid's stride.
inline unsigned grid_of(int64_t workgroups) {
  constexpr int64_t kMost = int64_t(1) << 22;
  return unsigned(workgroups < kMost ? workgroups : kMost);
}

}  // namespace net
}  // namespace gs
