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

// --- the gradient ------------------------------------------------------------------
//
// Positions of the sorted order are cut into stretches of `len`, so that an id
// of many rows and ids of one row each cost the same.  L lanes walk a stretch
// (C chunks of the row each, kAhead rows in flight) and write a table row
// wherever the id changes.  An id that reaches over a stretch's ends leaves a
// partial row there instead: part[stretch][0] for the id that began before,
// part[stretch][1] for the one that begins here and goes on.  k_join adds those
// up, stretch after stretch.  Rows of no id are filled with zeros by further
// workgroups of the first launch.

constexpr int kLongest = 128;      // positions of a stretch
constexpr int kSpan = 32;          // an id over more stretches than that is joined by a whole workgroup
constexpr int kJoinThreads = 1024;
constexpr int kZeroRows = 8;       // table rows that L lanes look at

struct Stretches {
  float* part;
  int64_t count;
  int32_t len, slices;      // slices: of 64 C chunks, across the row
};

// The row at a sorted position and its table row; -1: none.
__device__ __forceinline__ int32_t row_at(const EmbedArgs& a, int64_t p) {
  const int32_t r = a.order[p];
  return r >= 0 && r < a.rows ? r : -1;
}
__device__ __forceinline__ int32_t key_at(const EmbedArgs& a, int32_t r) {
  if (r < 0) return -1;
  const int64_t id = id_at(a.ids, a.id_bytes, r);
  return id >= 0 && id < a.num_rows ? int32_t(id) : -1;
}
// Positions that belong to an id.
__device__ __forceinline__ int64_t positions(const EmbedArgs& a) {
  const int64_t n = a.offsets[a.num_rows];
  return n < 0 ? 0 : (n < a.rows ? n : a.rows);
}

template <typename T, typename O, int L, int C>
__global__ __launch_bounds__(kThreads) void k_sum(EmbedArgs a, Stretches s, int64_t sum_groups) {
  constexpr int K = kChunk<T>, kGroups = kThreads / L, kAhead = 8 / C < 2 ? 2 : 8 / C;
  __shared__ int32_t s_row[kGroups * kLongest];
  __shared__ int32_t s_key[kGroups * kLongest + 2];      // one position more on either side
  const Row<T> row(a.width);
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  if (int64_t(blockIdx.x) >= sum_groups) {
    // rows of no id
    const int64_t v0 = ((int64_t(blockIdx.x) - sum_groups) * kGroups + g) * kZeroRows;
    int64_t ends[kZeroRows + 1];
#pragma unroll
    for (int k = 0; k <= kZeroRows; ++k) ends[k] = a.offsets[std::min<int64_t>(v0 + k, a.num_rows)];
    const float none[K] = {};
#pragma unroll
    for (int k = 0; k < kZeroRows; ++k)
      if (v0 + k < a.num_rows && ends[k] == ends[k + 1])
        for (int c = l; c < row.chunks; c += L) row.store(static_cast<O*>(a.dtable) + (v0 + k) * a.lddt, c, none);
    return;
  }
  const int64_t n = positions(a), block = blockIdx.x / s.slices;
  const int slice = int(blockIdx.x - block * s.slices);
  const int64_t base = block * kGroups * s.len;
  if (base >= n) return;
  for (int i = threadIdx.x; i < kGroups * s.len + 2; i += kThreads) {
    const int64_t p = base - 1 + i;
    const int32_t r = p >= 0 && p < n ? row_at(a, p) : -1;
    s_key[i] = p < 0 || p >= n ? -2 : key_at(a, r);
    if (i >= 1 && i <= kGroups * s.len) s_row[i - 1] = r;
  }
  __syncthreads();
  const int first = g * s.len;
  const int end = int(std::min<int64_t>(first + s.len, n - base));
  if (first >= end) return;
  int c[C];
#pragma unroll
  for (int j = 0; j < C; ++j) c[j] = slice * (L * C) + j * L + l;
  float sum[C][K] = {};
  float* const part = s.part + (block * kGroups + g) * 2 * a.width;
  O* const dtable = static_cast<O*>(a.dtable);
  int32_t key = s_key[first + 1];
  bool head = s_key[first] == key;
  auto flush = [&](bool partial, int which) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (c[j] < row.chunks) {
        if (partial) {
          row.store(part + which * a.width, c[j], sum[j]);
        } else if (key >= 0) {
          float o[K];
#pragma unroll
          for (int i = 0; i < K; ++i) o[i] = sum[j][i] * a.scale;
          row.store(dtable + key * a.lddt, c[j], o);
        }
      }
#pragma unroll
      for (int i = 0; i < K; ++i) sum[j][i] = 0.0f;
    }
  };
  for (int p = first; p < end; p += kAhead) {
    Chunk<T> x[kAhead][C];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int32_t r = p + u < end ? s_row[p + u] : -1;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        x[u][j] = Chunk<T>{};
        if (r >= 0 && c[j] < row.chunks) x[u][j] = row.load(static_cast<const T*>(a.dy) + r * a.lddy, c[j]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (p + u >= end) break;
      const int32_t k = s_key[p + u + 1];
      if (k != key) {
        flush(head, 0);
        key = k;
        head = false;
      }
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < K; ++i) sum[j][i] += float(x[u][j].v[i]);
    }
  }
  const bool on = s_key[end + 1] == key;
  flush(head || on, head ? 0 : 1);
}

// Partial rows to table rows.  The first workgroups: L lanes for each stretch
// whose last id begins there and goes on over at most kSpan further ones.  The
// others: a workgroup for every kSpan stretches and 64 columns; the one id that
// reaches over their end, if it is longer than that and begins there.
template <typename O, int L>
__global__ __launch_bounds__(kJoinThreads) void k_join(EmbedArgs a, Stretches s, int64_t short_groups) {
  constexpr int kGroups = kJoinThreads / L;
  __shared__ float box[kJoinThreads / 64][64];
  const Row<float> row(a.width);
  const int64_t n = positions(a), used = (n + s.len - 1) / s.len;
  if (int64_t(blockIdx.x) < short_groups) {
    const int64_t st = int64_t(blockIdx.x) * kGroups + threadIdx.x / L;
    const int64_t p0 = st * s.len, p1 = p0 + s.len;
    if (p1 >= n) return;
    const int32_t k0 = key_at(a, row_at(a, p0)), k1 = key_at(a, row_at(a, p1 - 1)), k2 = key_at(a, row_at(a, p1));
    const int32_t before = p0 > 0 ? key_at(a, row_at(a, p0 - 1)) : -2;
    if (k1 < 0 || k1 != k2 || (k0 == k1 && before == k1)) return;
    const int64_t last = std::min<int64_t>((std::max<int64_t>(a.offsets[k1 + 1], p1 + 1) - 1) / s.len, used - 1);
    if (last - st > kSpan) return;
    for (int c = threadIdx.x % L; c < row.chunks; c += L) {
      Chunk<float> x = row.load(s.part + (st * 2 + 1) * a.width, c);
      float sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = x.v[i];
#pragma unroll 4
      for (int64_t q = st + 1; q <= last; ++q) {
        x = row.load(s.part + q * 2 * a.width, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += x.v[i];
      }
      O* const dst = static_cast<O*>(a.dtable) + k1 * a.lddt;
      if (a.width >= 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[row.at(c) + i] = O(sum[i] * a.scale);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < a.width) dst[i] = O(sum[i] * a.scale);
      }
    }
    return;
  }
  const int across = (a.width + 63) / 64;
  const int64_t block = (int64_t(blockIdx.x) - short_groups) / across;
  const int col = int((int64_t(blockIdx.x) - short_groups) - block * across) * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  const int64_t p = (block + 1) * kSpan * s.len;
  if (p >= n) return;      // the whole workgroup, as below
  const int32_t k = key_at(a, row_at(a, p));
  if (k < 0 || k != key_at(a, row_at(a, p - 1))) return;
  const int64_t begin = std::max<int64_t>(a.offsets[k], 0) / s.len;
  const int64_t last = std::min<int64_t>((std::max<int64_t>(a.offsets[k + 1], 1) - 1) / s.len, used - 1);
  if (last - begin <= kSpan || begin < block * kSpan || begin >= (block + 1) * kSpan) return;
  float sum = 0.0f;
  if (col < a.width) {
    if (w == 0) sum = s.part[(begin * 2 + 1) * a.width + col];
#pragma unroll 16
    for (int64_t q = begin + 1 + w; q <= last; q += kJoinThreads / 64) sum += s.part[q * 2 * a.width + col];
  }
  box[w][threadIdx.x & 63] = sum;
  __syncthreads();
  if (w != 0 || col >= a.width) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 64; ++i) sum += box[i][threadIdx.x];
  static_cast<O*>(a.dtable)[k * a.lddt + col] = O(sum * a.scale);
}

template <typename T, int L>
hipError_t go_fwd(const EmbedArgs& a, hipStream_t st) {
  k_lookup<T, L><<<grid_of((a.rows + kThreads / L - 1) / (kThreads / L)), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

// Lanes and chunks of a lane that walk a stretch.
struct Shape {
  int lanes, each, slices;
};
Shape shape_of(int chunks) {
  if (chunks <= 64) return {row_lanes(chunks), 1, 1};
  const int each = std::min((chunks + 63) / 64, 4);
  return {64, each, (chunks + 64 * each - 1) / (64 * each)};
}

// Stretches are as long as 8192 waves (8 for each SIMD) leave them, 8 to
// kLongest positions: longer ones leave fewer partial rows.
Stretches stretches_of(int type, int64_t rows, int32_t width, void* ws) {
  const int chunk = type == kTypeF32 ? 4 : 8;
  const Shape f = shape_of((width + chunk - 1) / chunk);
  int32_t len = 8;
  while (len < kLongest && rows * f.slices * f.lanes > int64_t(len) * 64 * 8192) len *= 2;
  return {static_cast<float*>(ws), (rows + len - 1) / len, len, f.slices};
}

template <typename T, typename O, int L, int C>
void go_sum(const EmbedArgs& a, const Stretches& s, hipStream_t st) {
  constexpr int kGroups = kThreads / L;
  const int64_t sums = (s.count + kGroups - 1) / kGroups * s.slices;
  const int64_t zeros = (a.num_rows + kGroups * kZeroRows - 1) / (kGroups * kZeroRows);
  k_sum<T, O, L, C><<<unsigned(sums + zeros), kThreads, 0, st>>>(a, s, sums);
}

template <typename O, int L>
void go_join(const EmbedArgs& a, const Stretches& s, hipStream_t st) {
  if (s.count < 2) return;
  const int64_t spans = (s.count + kJoinThreads / L - 1) / (kJoinThreads / L);
  const int64_t longs = s.count > kSpan ? (s.count + kSpan - 1) / kSpan * ((a.width + 63) / 64) : 0;
  k_join<O, L><<<unsigned(spans + longs), kJoinThreads, 0, st>>>(a, s, spans);
}

template <typename T, typename O>
hipError_t embed_bwd(int type, const EmbedArgs& a, void* ws, hipStream_t st) {
  const Shape f = shape_of((a.width + kChunk<T> - 1) / kChunk<T>);
  const Stretches s = stretches_of(type, a.rows, a.width, ws);
  if (f.lanes == 8)
    go_sum<T, O, 8, 1>(a, s, st);
  else if (f.lanes == 16)
    go_sum<T, O, 16, 1>(a, s, st);
  else if (f.lanes == 32)
    go_sum<T, O, 32, 1>(a, s, st);
  else if (f.each == 1)
    go_sum<T, O, 64, 1>(a, s, st);
  else if (f.each == 2)
    go_sum<T, O, 64, 2>(a, s, st);
  else if (f.each == 3)
    go_sum<T, O, 64, 3>(a, s, st);
  else
    go_sum<T, O, 64, 4>(a, s, st);
  if (a.width <= 64)
    go_join<O, 16>(a, s, st);
  else
    go_join<O, 64>(a, s, st);
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

}  // namespace
}  // namespace net

size_t embedding_bwd_ws_bytes(int type, int64_t rows, int64_t, int32_t width) {
  return size_t(net::stretches_of(type, rows, width, nullptr).count) * 2 * size_t(width) * sizeof(float);
}

hipError_t launch_embedding_fwd(int type, const EmbedArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return net::embed_fwd<net::bf16>(a, st);
  if (type == kTypeF16) return net::embed_fwd<net::f16>(a, st);
  return net::embed_fwd<float>(a, st);
}

hipError_t launch_embedding_bwd(int type, const EmbedArgs& a, void* ws, hipStream_t st) {
  if (type == kTypeF32) return net::embed_bwd<float, float>(type, a, ws, st);
  if (type == kTypeBF16)
    return a.dtable_f32 ? net::embed_bwd<net::bf16, float>(type, a, ws, st)
                        : net::embed_bwd<net::bf16, net::bf16>(type, a, ws, st);
  return a.dtable_f32 ? net::embed_bwd<net::f16, float>(type, a, ws, st)
                      : net::embed_bwd<net::f16, net::f16>(type, a, ws, st);
}

}  // namespace gs
