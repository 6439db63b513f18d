// Rows in 16-byte chunks for the operators that copy, scale and sum whole
// rows (embedding.hip, route.hip).
#pragma once

#include <algorithm>

#include "net_common.hpp"

namespace gs {
namespace net {

// A chunk as one vector: its elements one by one would be taken for loads of
// their own, and one of them put behind a branch.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ Chunk<T> load_whole(const T* __restrict__ p) {
  u32x4 w;
  __builtin_memcpy(&w, p, 16);
  return __builtin_bit_cast(Chunk<T>, w);
}

// kFar: past the caches, for an output that is larger than they are (is_far
// below), so that what else they hold stays.  (A branch would not do: of two
// stores that differ in nothing else the compiler makes one.)
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <bool kFar, typename T>
__device__ __forceinline__ void store_whole(T* __restrict__ p, const Chunk<T>& c) {
  if constexpr (kFar)
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, c), reinterpret_cast<u32x4_any*>(p));
  else
    store_chunk(p, c);
}

// A row of at least one chunk's width is covered by whole chunks, the last
// one moved back onto the row's end, so that no width takes a slower path:
// what two chunks share is read twice and written twice with the same values.
// kNarrow: a row of less than a chunk, its one chunk in part.  That is a
// template's choice and not a branch, because a load behind a branch is waited
// for before the next one is asked for.
template <typename T, bool kNarrow>
struct Row {
  static constexpr int K = kChunk<T>;
  int width, chunks;
  __device__ __forceinline__ explicit Row(int w) : width(w), chunks(kNarrow ? 1 : (w + K - 1) / K) {}
  __device__ __forceinline__ int at(int c) const {     // first column of chunk c
    return kNarrow ? 0 : std::min(c * K, width - K);
  }
  __device__ __forceinline__ int again(int c) const {  // its columns that the chunk before has too
    return c * K - at(c);
  }
  __device__ __forceinline__ Chunk<T> load(const T* __restrict__ row, int c) const {
    if constexpr (kNarrow)
      return load_chunk_n(row, width);
    else
      return load_whole(row + at(c));
  }
  template <bool kFar>
  __device__ __forceinline__ void copy(T* __restrict__ row, int c, const Chunk<T>& v) const {
    if constexpr (kNarrow)
      store_chunk_n(row, v, width);
    else
      store_whole<kFar>(row + at(c), v);
  }
  template <bool kFar = false, typename O>      // O of T's size, or fp32 for 16-bit T
  __device__ __forceinline__ void store(O* __restrict__ row, int c, const float (&v)[K]) const {
    if constexpr (kNarrow) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (i < width) row[i] = O(v[i]);
    } else {
      constexpr int kPart = kChunk<O>;
#pragma unroll
      for (int h = 0; h < K; h += kPart) {
        Chunk<O> o;
#pragma unroll
        for (int i = 0; i < kPart; ++i) o.v[i] = O(v[h + i]);
        store_whole<kFar>(row + at(c) + h, o);
      }
    }
  }
  // Without the columns that the chunk before has too: what rows that are
  // read and written in place need.
  __device__ __forceinline__ void store_rest(T* __restrict__ row, int c, const float (&v)[K]) const {
    if (kNarrow || again(c) == 0) {
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

// Whether an output of whole 16-byte chunks is larger than the cache beside
// the memory (256 MB).  Lookup of 1,000,000 x 256 bf16, whose table of 51 MB then
// stays in that cache: 155 -> 143 us; 400,000 x 256 bf16 to two places: 128 -> 124.
// Rows that begin inside a chunk take longer (50,021 x 515 fp32 47 -> 55).
inline bool is_far(const void* p, int64_t ld, int64_t rows, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem % 16 == 0 && rows * ld * int64_t(elem) >= int64_t(1) << 28;
}

// A launch takes less than 2^32 threads: kernels whose items may be more walk
// them with the grid's stride.
inline unsigned grid_of(int64_t workgroups) {
  constexpr int64_t kMost = int64_t(1) << 22;
  return unsigned(workgroups < kMost ? workgroups : kMost);
}

}  // namespace net
}  // namespace gs
