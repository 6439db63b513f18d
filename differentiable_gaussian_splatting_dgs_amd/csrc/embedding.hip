// Rows looked up in a table, and the table's gradient by sorted ids.
//
//   forward   y[i] = scale table[id[i]], zeros for an id outside the table
//   backward  dtable[v] = scale sum of dy[i] over id[i] = v
//
// Both are bound by the bytes of the rows.  Sums are fp32; the rounding into
// the storage type is the last step.  1,000,000 x 256 bf16 from and to 100,000
// rows: lookup 143 us (512 MB written, 470 MB of the table read again from
// beyond the L2: 6.9 TB/s); gradient 133 us for the sums (575 MB read, of rows
// in any order: a gather of whole rows reaches 5.0 TB/s) and 9 for the joins,
// behind 54 of the sort.
#include <algorithm>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t id_at(const void* __restrict__ ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// Chunk c of N rows from r0 on.  Nothing here is behind a branch, so that the
// ids, and then the chunks, are in flight together.
template <typename T, typename I, int N, bool kFar, bool kNarrow>
__device__ __forceinline__ void look_up(const EmbedArgs& a, const Row<T, kNarrow>& row, int64_t r0, int c) {
  constexpr int K = kChunk<T>;
  int64_t id[N];
#pragma unroll
  for (int u = 0; u < N; ++u) id[u] = static_cast<const I*>(a.ids)[r0 + u];
  Chunk<T> x[N];
  bool there[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    there[u] = id[u] >= 0 && id[u] < a.num_rows;
    x[u] = row.load(static_cast<const T*>(a.table) + (there[u] ? id[u] : 0) * a.ldt, c);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    float v[K];
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = there[u] ? float(x[u].v[i]) * a.scale : 0.0f;
    row.template store<kFar>(static_cast<T*>(a.y) + (r0 + u) * a.ldy, c, v);
  }
}

// Items are slices of kRows rows: L lanes, a chunk of each row for each lane.
// A row alone waits for its id and then for its chunk, and as many waves as
// fit do not make up for that: several rows at a time where there are many.
template <typename T, typename I, int L, int kRows, bool kFar, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_lookup(EmbedArgs a, int slices, int64_t items) {
  constexpr int kGroups = kThreads / L;
  const Row<T, kNarrow> row(a.width);
  for (int64_t item = int64_t(blockIdx.x) * kGroups + threadIdx.x / L; item < items;
       item += int64_t(gridDim.x) * kGroups) {
    const int64_t part = item / slices, r0 = part * kRows;
    const int c = int(item - part * slices) * L + threadIdx.x % L;
    if (c >= row.chunks) continue;
    if (kRows == 1 || r0 + kRows <= a.rows)
      look_up<T, I, kRows, kFar>(a, row, r0, c);
    else
      for (int64_t r = r0; r < a.rows; ++r) look_up<T, I, 1, kFar>(a, row, r, c);
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
constexpr int kZeroRows = 8;       // table rows that L lanes look at

struct Stretches {
  float* part;
  int32_t* goes_on;         // the id that begins in a stretch and goes on behind it, or -1
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

template <typename T, typename O, int L, int C, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_sum(EmbedArgs a, Stretches s, int64_t sum_groups) {
  constexpr int K = kChunk<T>, kGroups = kThreads / L, kAhead = 8 / C < 2 ? 2 : 8 / C;
  __shared__ int32_t s_row[kGroups * kLongest];
  __shared__ int32_t s_key[kGroups * kLongest + 2];      // one position more on either side
  const Row<T, kNarrow> row(a.width);
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  if (int64_t(blockIdx.x) >= sum_groups) {
    // rows of no id
    const float none[K] = {};
    for (int64_t v0 = ((int64_t(blockIdx.x) - sum_groups) * kGroups + g) * kZeroRows; v0 < a.num_rows;
         v0 += (int64_t(gridDim.x) - sum_groups) * kGroups * kZeroRows) {
      int64_t ends[kZeroRows + 1];
#pragma unroll
      for (int k = 0; k <= kZeroRows; ++k) ends[k] = a.offsets[std::min<int64_t>(v0 + k, a.num_rows)];
#pragma unroll
      for (int k = 0; k < kZeroRows; ++k)
        if (v0 + k < a.num_rows && ends[k] == ends[k + 1])
          for (int c = l; c < row.chunks; c += L) row.store(static_cast<O*>(a.dtable) + (v0 + k) * a.lddt, c, none);
    }
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
      // past the end, and of no row: any row, whose sum is not used
      const int32_t r = std::max(s_row[std::min(p + u, end - 1)], 0);
#pragma unroll
      for (int j = 0; j < C; ++j)
        x[u][j] = row.load(static_cast<const T*>(a.dy) + r * a.lddy, std::min(c[j], row.chunks - 1));
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
  if (slice == 0 && l == 0) s.goes_on[block * kGroups + g] = on && !head ? key : -1;
  flush(head || on, head ? 0 : 1);
}

// Partial rows to table rows.  The first workgroups: L lanes for each stretch
// whose last id begins there and goes on over at most kSpan further ones.  The
// others: a workgroup for every kSpan stretches and 64 columns; of the ids that
// begin in them only the last can be longer than that.
template <typename O, int L, bool kNarrow>
__global__ __launch_bounds__(kThreads) void k_join(EmbedArgs a, Stretches s, int64_t short_groups) {
  constexpr int kGroups = kThreads / L, kWaves = kThreads / 64;
  __shared__ float box[kWaves][64];
  const Row<float, kNarrow> row(a.width);
  const int64_t n = positions(a), used = (n + s.len - 1) / s.len;
  // the last stretch of an id that goes on behind stretch st
  auto last_of = [&](int32_t key, int64_t st) {
    const int64_t end = std::min(a.offsets[key + 1], n);
    return std::max(st, (std::max<int64_t>(end, 1) - 1) / s.len);
  };
  if (int64_t(blockIdx.x) < short_groups) {
    const int64_t st = int64_t(blockIdx.x) * kGroups + threadIdx.x / L;
    const int32_t key = st < used ? s.goes_on[st] : -1;
    if (key < 0) return;
    const int64_t last = last_of(key, st);
    if (last - st > kSpan) return;
    O* const dst = static_cast<O*>(a.dtable) + key * a.lddt;
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
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row.at(c) + i < a.width) dst[row.at(c) + i] = O(sum[i] * a.scale);
    }
    return;
  }
  const int across = (a.width + 63) / 64, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t block = (int64_t(blockIdx.x) - short_groups) / across;
  const int col = int((int64_t(blockIdx.x) - short_groups) - block * across) * 64 + lane;
  const int64_t mine = block * kSpan + lane;
  const int32_t id = lane < kSpan && mine < used ? s.goes_on[mine] : -1;
  const uint64_t begins = __ballot(id >= 0);
  if (begins == 0) return;      // the whole workgroup, as below
  const int top = 63 - __builtin_clzll(begins);
  const int64_t st = block * kSpan + top;
  const int32_t key = __shfl(id, top, 64);
  const int64_t last = last_of(key, st);
  if (last - st <= kSpan) return;
  float sum = 0.0f;
  if (col < a.width) {
    if (w == 0) sum = s.part[(st * 2 + 1) * a.width + col];
#pragma unroll 16
    for (int64_t q = st + 1 + w; q <= last; q += kWaves) sum += s.part[q * 2 * a.width + col];
  }
  box[w][lane] = sum;
  __syncthreads();
  if (w != 0 || col >= a.width) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) sum += box[i][lane];
  static_cast<O*>(a.dtable)[key * a.lddt + col] = O(sum * a.scale);
}

template <typename T, typename I, int L, bool kNarrow = false>
hipError_t go_fwd(const EmbedArgs& a, hipStream_t st) {
  constexpr int kGroups = kThreads / L, kRows = 4;
  const int slices = ((a.width + kChunk<T> - 1) / kChunk<T> + L - 1) / L;
  // several rows where that leaves 16 waves for each SIMD
  const int64_t items = (a.rows + kRows - 1) / kRows * slices, ones = a.rows * slices;
  if (items * L < 64 * 16384)
    k_lookup<T, I, L, 1, false, kNarrow><<<grid_of((ones + kGroups - 1) / kGroups), kThreads, 0, st>>>(a, slices, ones);
  else if (is_far(a.y, a.ldy, a.rows, sizeof(T)))
    k_lookup<T, I, L, kRows, true, kNarrow>
        <<<grid_of((items + kGroups - 1) / kGroups), kThreads, 0, st>>>(a, slices, items);
  else
    k_lookup<T, I, L, kRows, false, kNarrow>
        <<<grid_of((items + kGroups - 1) / kGroups), kThreads, 0, st>>>(a, slices, items);
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

// Stretches are as long as 4096 waves (4 for each SIMD) leave them, 8 to
// kLongest positions: longer ones leave fewer partial rows, but 8,191 rows are
// too few for them (1,000,000 x 256 bf16 with 128 positions 200 us, 64 208, 32 212,
// 16 233; 8,191 x 515 fp32 with 8 44 us, 32 50, 128 94).
Stretches stretches_of(int type, int64_t rows, int32_t width, void* ws) {
  const int chunk = type == kTypeF32 ? 4 : 8;
  const Shape f = shape_of((width + chunk - 1) / chunk);
  int32_t len = 8;
  while (len < kLongest && rows * f.slices * f.lanes > int64_t(len) * 64 * 4096) len *= 2;
  Stretches s{nullptr, nullptr, (rows + len - 1) / len, len, f.slices};
  s.goes_on = static_cast<int32_t*>(ws);
  s.part = reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(size_t(s.count) * 4, 256));
  return s;
}
size_t stretches_bytes(const Stretches& s, int32_t width) {
  return align_up(size_t(s.count) * 4, 256) + size_t(s.count) * 2 * size_t(width) * sizeof(float);
}

template <typename T, typename O, int L, int C, bool kNarrow = false>
void go_sum(const EmbedArgs& a, const Stretches& s, hipStream_t st) {
  constexpr int kGroups = kThreads / L;
  const int64_t sums = (s.count + kGroups - 1) / kGroups * s.slices;
  const int64_t zeros = grid_of((a.num_rows + kGroups * kZeroRows - 1) / (kGroups * kZeroRows));
  k_sum<T, O, L, C, kNarrow><<<unsigned(sums + zeros), kThreads, 0, st>>>(a, s, sums);
}

template <typename O, int L, bool kNarrow = false>
void go_join(const EmbedArgs& a, const Stretches& s, hipStream_t st) {
  if (s.count < 2) return;
  const int64_t spans = (s.count + kThreads / L - 1) / (kThreads / L);
  const int64_t longs = s.count > kSpan ? (s.count + kSpan - 1) / kSpan * ((a.width + 63) / 64) : 0;
  k_join<O, L, kNarrow><<<unsigned(spans + longs), kThreads, 0, st>>>(a, s, spans);
}

template <typename T, typename O>
hipError_t embed_bwd(int type, const EmbedArgs& a, void* ws, hipStream_t st) {
  const Shape f = shape_of((a.width + kChunk<T> - 1) / kChunk<T>);
  const Stretches s = stretches_of(type, a.rows, a.width, ws);
  if (a.width < kChunk<T>)
    go_sum<T, O, 8, 1, true>(a, s, st);
  else if (f.lanes == 8)
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
  if (a.width < 4)
    go_join<O, 16, true>(a, s, st);
  else if (a.width <= 64)
    go_join<O, 16>(a, s, st);
  else
    go_join<O, 64>(a, s, st);
  return hipGetLastError();
}

template <typename T, typename I>
hipError_t embed_fwd(const EmbedArgs& a, hipStream_t st) {
  if (a.width < kChunk<T>) return go_fwd<T, I, 2, true>(a, st);
  const int chunks = (a.width + kChunk<T> - 1) / kChunk<T>;
  // 1,000,000 x 16 bf16 with 8 lanes 16 us, with 2 12
  if (chunks <= 2) return go_fwd<T, I, 2>(a, st);
  if (chunks <= 4) return go_fwd<T, I, 4>(a, st);
  switch (row_lanes(chunks)) {
    case 8: return go_fwd<T, I, 8>(a, st);
    case 16: return go_fwd<T, I, 16>(a, st);
    case 32: return go_fwd<T, I, 32>(a, st);
    default: return go_fwd<T, I, 64>(a, st);
  }
}

}  // namespace
}  // namespace net

size_t embedding_bwd_ws_bytes(int type, int64_t rows, int64_t, int32_t width) {
  return net::stretches_bytes(net::stretches_of(type, rows, width, nullptr), width);
}

template <typename I>
static hipError_t embed_fwd_of(int type, const EmbedArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return net::embed_fwd<net::bf16, I>(a, st);
  if (type == kTypeF16) return net::embed_fwd<net::f16, I>(a, st);
  return net::embed_fwd<float, I>(a, st);
}

hipError_t launch_embedding_fwd(int type, const EmbedArgs& a, hipStream_t st) {
  return a.id_bytes == 4 ? embed_fwd_of<int32_t>(type, a, st) : embed_fwd_of<int64_t>(type, a, st);
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
