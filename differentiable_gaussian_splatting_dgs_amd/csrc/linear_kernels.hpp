// The linear layer's kernels, included by linear_bf16.hip, linear_f16.hip and
// linear_f32.hip (one storage type each, so that they build side by side).
//
//   forward    z = x w^T + bias, y = act(z) + residual
//   backward   dz = dy act'(z); dx = dz w; dw = dz^T x; db = sum of dz's rows
//
// One tiled product C[m][n] = sum_k A(m, k) B(n, k) serves the three:
//   kFwd  m = rows, n = out, k = in    A = x  (k along memory), B = w (k along memory)
//   kDx   m = rows, n = in,  k = out   A = dz (k along memory), B = w (n along memory)
//   kDw   m = out,  n = in,  k = rows  A = dz (m along memory), B = x (n along memory)
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "net_common.hpp"

namespace gs {
namespace net {
namespace {

enum Mode { kFwd = 0, kDx = 1, kDw = 2 };

struct ProductArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb, b_group;      // b_group: elements from one group's weights to the next
  const int64_t* offsets;
  int32_t rows, groups;           // groups == 0: one group of all rows
  int32_t m, n, k;                // the fixed extents (kFwd, kDx: m unused; kDw: k unused)
  int32_t unit;                   // kDw: rows of a stretch; else the tile height
  int32_t tiles_n, tiles;         // tiles across, tiles in all (kDw: tiles of one stretch)
  // epilogue
  const float* bias;
  const void* residual;
  void* out;
  void* z;
  float* part;                    // kDw: partial products, one plane of `plane` values per stretch: [m][n], then [m] of db
  float* db;                      // kDw: the sums of a's columns, or NULL
  int64_t plane;
  int64_t ldr, ldo, ldz;
  int32_t act, out_f32;
};

// --- matrix instructions ------------------------------------------------------------

// A fragment is 16 bytes of one row along k: lane l holds row l % 16 and
// k-chunk l / 16 of a 16 x (64 bytes) block.  16-bit types: one 16x16x32
// instruction; fp32: four 16x16x4, component c of every lane's chunk in the
// c-th (`part`; the same order of k on both sides, so the sum is the same).
// D: lane l holds rows 4 (l / 16) .. + 3 of column l % 16.
template <typename T>
struct Frag;
template <>
struct Frag<bf16> {
  typedef __bf16 V __attribute__((ext_vector_type(8)));
  static constexpr int kParts = 1;
  static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<f16> {
  typedef _Float16 V __attribute__((ext_vector_type(8)));
  static constexpr int kParts = 1;
  static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  typedef float V __attribute__((ext_vector_type(4)));
  static constexpr int kParts = 4;
  static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c, int part) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a[part], b[part], c, 0, 0, 0);
  }
};

// All pairs of a step's fragments; the parts of one pair, which wait for each
// other, lie as far apart as they can.
template <typename T, int FM, int FN>
__device__ __forceinline__ void mma_all(const typename Frag<T>::V (&fb)[FN], const typename Frag<T>::V (&fa)[FM],
                                        f32x4 (&acc)[FM][FN]) {
#pragma unroll
  for (int c = 0; c < Frag<T>::kParts; ++c)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = Frag<T>::mma(fb[j], fa[i], acc[i][j], c);
}

// --- tiles in LDS ---------------------------------------------------------------------

// A k step is KB = 128 bytes of k (64 16-bit or 32 fp32 values), or 64 where
// the tiles come straight from memory.  Two layouts of a D-row operand, both
// of D * KB bytes:
//   along k    [D][KB bytes]: the chunks of row r permuted by r so that the 8
//              rows of a 128-byte LDS access lie on different banks
//   across k   [k][D]: read back transposed, 16-bit types with the LDS
//              transpose read (4 x 16 blocks), fp32 value by value; the
//              chunks of row k are permuted in pairs (16-bit) or fours
//              (fp32) by the bits of k that a wave's read spans
template <typename T>
constexpr int kStep = int(128 / sizeof(T));

template <typename T, int D>
__device__ __forceinline__ int across_swizzle(int k) {
  constexpr int chunks = D / kChunk<T>;
  if constexpr (sizeof(T) == 2)
    return (2 * ((k & 3) | ((k >> 1) & 4))) & (chunks - 1);
  else
    return (((k >> 2) & 3) << 2) & (chunks - 1);
}

template <int KB>
__device__ __forceinline__ int along_swizzle(int r) {
  return KB == 128 ? r & 7 : (r >> 1) & 3;
}

// Byte offset of chunk c of row r.
template <typename T, int D, bool ACROSS, int KB = 128>
__device__ __forceinline__ int tile_at(int r, int c) {
  if constexpr (ACROSS)
    return (r * (D / kChunk<T>) + (c ^ across_swizzle<T, D>(r))) * 16;
  else
    return (r * (KB / 16) + (c ^ along_swizzle<KB>(r))) * 16;
}

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// The fragment of rows d0 .. d0 + 15, k chunk group kk (64 bytes of k).
template <typename T, int D, bool ACROSS, int KB = 128>
__device__ __forceinline__ typename Frag<T>::V read_frag(const char* tile, int d0, int kk, int lane) {
  using V = typename Frag<T>::V;
  const int i = lane & 15, g = lane >> 4;
  if constexpr (!ACROSS) {
    return *reinterpret_cast<const V*>(tile + tile_at<T, D, false, KB>(d0 + i, 4 * kk + g));
  } else if constexpr (sizeof(T) == 2) {
    // lane i of a quarter wave reads 4 values of row k + i / 4 at column
    // 4 (i % 4); the read hands it column i of the four rows
    s16x8 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 32 * kk + 8 * g + 4 * h + (i >> 2);
      const char* p = tile + tile_at<T, D, true>(k, (d0 >> 3) + ((i & 3) >> 1)) + (i & 1) * 8;
      const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
      v[4 * h] = u[0];
      v[4 * h + 1] = u[1];
      v[4 * h + 2] = u[2];
      v[4 * h + 3] = u[3];
    }
    return __builtin_bit_cast(V, v);
  } else {
    V v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = 16 * kk + 4 * g + c;
      v[c] = *reinterpret_cast<const float*>(tile + tile_at<T, D, true>(k, (d0 + i) >> 2) + ((d0 + i) & 3) * 4);
    }
    return v;
  }
}

// Transposed fragments of a tile that lies along k, [step][ROWS][128 bytes]
// (16-bit types): columns d0 .. d0 + 15 over rows 32 kk ...  Of the chunk
// address c ^ (r % 8) a lane's own bits are few: with c = 2 jj + b (jj the 16
// columns within the step) and r % 8 = 4 h + q it is (b ^ (q & 1)) + 2 (jj ^ 2 h
// ^ (q >> 1)), so four lane addresses, one for each jj ^ 2 h, serve every
// fragment; the rest are constants of the instruction.
struct Across {
  uint32_t at[4];   // byte offsets from the tile
  // first: the 16 columns of the step that block 0 is (blocks j go on from
  // there by ^, which is + where a wave has first + j <= 3 blocks a step)
  __device__ __forceinline__ void init(int lane, int first) {
    const int i = lane & 15, g = lane >> 4, q = i >> 2;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      at[m] = uint32_t((8 * g + q) * 128 + ((((i & 3) >> 1) ^ (q & 1)) + 2 * (m ^ first ^ (q >> 1))) * 16 + (i & 1) * 8);
  }
  // j: block from the step that `tile` points at
  template <typename T, int ROWS>
  __device__ __forceinline__ typename Frag<T>::V read(const char* tile, int j, int kk) const {
    s16x8 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(tile + at[(j & 3) ^ (2 * h)] + ((j >> 2) * ROWS * 128 + kk * 4096 + h * 512)));
      v[4 * h] = u[0];
      v[4 * h + 1] = u[1];
      v[4 * h + 2] = u[2];
      v[4 * h + 3] = u[3];
    }
    return __builtin_bit_cast(typename Frag<T>::V, v);
  }
};

// Global -> registers -> LDS for one operand, at any alignment.  `rows` and
// `cols`: what is left of the operand from the tile's corner; values past
// them are 0 along k, and anything across it (in columns whose results are
// never stored).  Whole k steps load 16 bytes everywhere, unconditionally:
// rows past the end repeat the last one, and a chunk over a row's end reads on
// into the row that follows.  Only the last step has to look where the
// operand's memory ends (`mem` rows from the corner on).  `narrow`: rows of
// under 8 values, which no chunk fits.
template <typename T, int D, bool ACROSS, int THREADS>
struct Stage {
  static constexpr int kPer = D * 8 / THREADS;
  static constexpr int kAcross = ACROSS ? D / kChunk<T> : 8;   // chunks of a tile row
  Chunk<T> c[kPer];
  __device__ __forceinline__ void load(const T* __restrict__ p, int64_t ld, int rows, int cols, int mem, bool narrow,
                                       int tid) {
    if (!narrow && (ACROSS ? rows > kStep<T> : cols >= kStep<T>)) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int id = j * THREADS + tid, r = id / kAcross, at = (id % kAcross) * kChunk<T>;
        if constexpr (ACROSS)
          c[j] = load_chunk(p + int64_t(r) * ld + (at < cols ? at : 0));
        else
          c[j] = load_chunk(p + int64_t(r < rows ? r : rows - 1) * ld + at);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int id = j * THREADS + tid, r = id / kAcross, at = (id % kAcross) * kChunk<T>;
        const int left = r < rows ? cols - at : 0, n = left < 0 ? 0 : left;
        const bool safe = n >= kChunk<T> || (n > 0 && !narrow && r + 1 < mem);
        if (safe) c[j] = load_chunk(p + int64_t(r) * ld + at);
#pragma unroll
        for (int i = 0; i < kChunk<T>; ++i) c[j].v[i] = i < n ? c[j].v[i] : T(0.0f);
        if (!safe && n > 0) c[j] = load_chunk_n(p + int64_t(r) * ld + at, n);
      }
    }
  }
  __device__ __forceinline__ void store(char* tile, int tid) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int id = j * THREADS + tid;
      *reinterpret_cast<Chunk<T>*>(tile + tile_at<T, D, ACROSS>(id / kAcross, id % kAcross)) = c[j];
    }
  }
};

// Global -> LDS without registers, for operands of whole aligned chunks: the
// buffer load writes lane i's 16 bytes at 16 i of the wave's kilobyte, so the
// permutation of the chunks is done on the addresses.  Rows past the end
// lie past the buffer's size and read as 0; across k, columns past the end
// hold whatever follows in the row (their results are never stored).
template <typename T, int D, bool ACROSS, int THREADS, int KB>
struct Direct {
  static constexpr int kPer = D * KB / 16 / THREADS;
  static constexpr int kAcross = ACROSS ? D / kChunk<T> : KB / 16;
  static_assert(ACROSS || (THREADS / kAcross) % 8 == 0, "one chunk for all of a thread's rows");
  uint32_t off[kPer];
  int chunk;   // along k: the chunk of the row this thread fetches
  __device__ __forceinline__ void init(int64_t ld, int tid) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int id = j * THREADS + tid, r = id / kAcross;
      const int c = (id % kAcross) ^ (ACROSS ? across_swizzle<T, D>(r) : along_swizzle<KB>(r));
      off[j] = uint32_t(r) * uint32_t(ld * sizeof(T)) + uint32_t(c) * 16u;
      if (j == 0) chunk = c;
    }
  }
  // `rows`, `cols`: the operand's extent from p on, cols in whole chunks along
  // k; none of either: zeros.
  __device__ __forceinline__ void load(const T* p, int64_t ld, int rows, int cols, char* tile, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the buffer builtins
    constexpr int step = KB / int(sizeof(T)), most_rows = ACROSS ? step : D, most_cols = ACROSS ? D : step;
    const int r = rows < most_rows ? rows : most_rows, c = cols < most_cols ? cols : most_cols;
    // whole chunks: an aligned chunk that holds a value of the row lies inside its padding
    const int whole = (c + kChunk<T> - 1) / kChunk<T> * kChunk<T>;
    const uint32_t bytes = r > 0 && c > 0 ? uint32_t(((r - 1) * ld + whole) * int64_t(sizeof(T))) : 0u;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, bytes, 0x00020000);
    const bool past = !ACROSS && chunk * kChunk<T> >= cols;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(tile + j * THREADS * 16 + wave * 1024), 16,
          past ? 0xfffffff0u : off[j], 0, 0, 0);
#endif
  }
};

// All but the last LOADS of every wave's loads into LDS have landed and its
// reads of LDS are done, then the workgroup meets (a set of one wave has
// nobody to meet).
template <int WAVES, int LOADS = 0>
__device__ __forceinline__ void tile_barrier() {
  if constexpr (WAVES > 1)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
  else
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS) : "memory");
}
template <int WAVES>
__device__ __forceinline__ void stage_barrier() {
  if constexpr (WAVES > 1)
    __syncthreads();
  else
    wave_sync();
}

// --- epilogue -----------------------------------------------------------------------------

// Eight values of an output row, as chunks of storage.
template <typename T>
struct Eight {
  static constexpr int kParts = 8 / kChunk<T>;
  Chunk<T> c[kParts];
  __device__ __forceinline__ float get(int i) const { return float(c[i / kChunk<T>].v[i % kChunk<T>]); }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i / kChunk<T>].v[i % kChunk<T>] = T(v[i]);
  }
  // n values at p (n < 8 in the last columns only)
  __device__ __forceinline__ void load(const T* __restrict__ p, int n) {
#pragma unroll
    for (int h = 0; h < kParts; ++h) c[h] = load_chunk_n(p + h * kChunk<T>, n - h * kChunk<T>);
  }
  __device__ __forceinline__ void store(T* __restrict__ p, int n) const {
#pragma unroll
    for (int h = 0; h < kParts; ++h) store_chunk_n(p + h * kChunk<T>, c[h], n - h * kChunk<T>);
  }
};

template <typename T>
__device__ __forceinline__ void act_eight(float (&v)[8], int act) {   // act is uniform: one branch for the eight
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_apply<T>(v[i], kActRelu);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_apply<T>(v[i], kActSilu);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_apply<T>(v[i], kActGelu);
  }
}

template <typename T>
__device__ __forceinline__ void slope_eight(float (&v)[8], int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_slope<T>(v[i], kActRelu);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_slope<T>(v[i], kActSilu);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_slope<T>(v[i], kActGelu);
  }
}

// --- the product ------------------------------------------------------------------------------

// Consecutive workgroups go round the 8 XCDs, each with an L2 of its own:
// hand every XCD one contiguous share of the tiles instead.
__device__ __forceinline__ int xcd_tile(int id, int n) {
  const int x = id & 7, share = n >> 3, more = n & 7;
  return x * share + std::min(x, more) + (id >> 3);
}

// What one wave does with a k step in LDS.  `sums`: also adds the columns
// of a (a product with a row of ones: exact, in fp32).
template <typename T, int BM, int BN, bool A_ACROSS, bool B_ACROSS, int KB, int FM, int FN, int FS>
__device__ __forceinline__ void multiply_step(const char* ta, const char* tb, int am, int bn, int lane,
                                              f32x4 (&acc)[FM][FN], f32x4 (&sum)[FS], bool sums) {
#pragma unroll
  for (int kk = 0; kk < KB / 64; ++kk) {
    typename Frag<T>::V fa[FM], fb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = read_frag<T, BM, A_ACROSS, KB>(ta, am + 16 * i, kk, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = read_frag<T, BN, B_ACROSS, KB>(tb, bn + 16 * j, kk, lane);
    mma_all<T, FM, FN>(fb, fa, acc);
    if constexpr (FS == FM) {
      if (sums) {
        typename Frag<T>::V one;
#pragma unroll
        for (int c = 0; c < kChunk<T>; ++c) one[c] = T(1.0f);
#pragma unroll
        for (int c = 0; c < Frag<T>::kParts; ++c)
#pragma unroll
          for (int i = 0; i < FM; ++i) sum[i] = Frag<T>::mma(one, fa[i], sum[i], c);
      }
    }
  }
}

// How the tiles that come straight from memory are staged: dw's smaller tiles,
// whose transposed reads leave the loads less time, in four half steps of 64
// bytes of k (64 heads of 512 x 512 over 131,072 rows in 128 x 128: 137 us against
// 147), the others in two whole steps, with half the barriers (16384 x 4096 x
// 4096 fp16, 256 x 256: forward 497 us against 510, dw 569 against 643).
constexpr bool half_steps(Mode mode, int bm) { return mode == kDw && bm < 256; }

// BM x BN outputs a workgroup, WM x WN waves.  The n side is the first
// operand of the matrix instruction, so that a lane's four results are
// neighbours along n; each wave then turns 16 rows at a time through LDS
// into whole chunks of output rows.  DIRECT: both operands in whole aligned
// chunks, loaded straight into the LDS stages ahead of the one that is
// multiplied; else through registers, at any alignment.  KW > 1: so many sets
// of WM x WN waves take the k steps in turn, for products of few tiles and a
// long k, whose time is the steps that wait on each other; the first set adds
// the others' results.
template <typename T, Mode MODE, int BM, int BN, int WM, int WN, bool DIRECT, int KW>
__device__ __forceinline__ void product_tile(const ProductArgs& p, int tile, char* lds) {
  constexpr int THREADS = 64 * WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr bool A_ACROSS = MODE == kDw, B_ACROSS = MODE != kFwd;
  constexpr int kPatch = TN + 4;   // floats of a patch row: 4 more keep its 16-byte writes off each other's banks
  const int set = KW > 1 ? __builtin_amdgcn_readfirstlane(int(threadIdx.x) / THREADS) : 0;
  const int tid = KW > 1 ? int(threadIdx.x) % THREADS : int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  char* const base = lds;
  constexpr bool kHalf = DIRECT && half_steps(MODE, BM);
  constexpr int kStages = kHalf ? 4 : 2, kB = kHalf ? 64 : 128;
  if (KW > 1) lds += set * (BM + BN) * kB * (DIRECT ? kStages : 1);

  // Which tile.  kFwd, kDx: the height index picks group and rows; kDw: the
  // stretch does (without planes to join, every group is one stretch, and
  // empty ones store their zeros), the tile inside the plane is apart from it.
  const int stretch = MODE == kDw ? tile / p.tiles : tile / p.tiles_n;
  const int within = MODE == kDw ? tile % p.tiles : tile % p.tiles_n;
  const Span s = MODE == kDw && p.part == nullptr ? group_span(p.offsets, p.groups, p.rows, p.unit, stretch)
                                                  : find_span(p.offsets, p.groups, p.rows, p.unit, stretch);
  if (s.e < 0) return;
  const int m0 = MODE == kDw ? within / p.tiles_n * BM : 0;
  const int n0 = (MODE == kDw ? within % p.tiles_n : within) * BN;
  const int m_left = MODE == kDw ? p.m - m0 : s.row1 - s.row0, n_left = p.n - n0;
  const int k_all = MODE == kDw ? s.row1 - s.row0 : p.k;
  const T* a = static_cast<const T*>(p.a) + int64_t(s.row0) * p.lda + m0;
  const T* b = static_cast<const T*>(p.b);
  if constexpr (MODE == kFwd) b += int64_t(s.e) * p.b_group + int64_t(n0) * p.ldb;
  if constexpr (MODE == kDx) b += int64_t(s.e) * p.b_group + n0;
  if constexpr (MODE == kDw) b += int64_t(s.row0) * p.ldb + n0;
  constexpr int kK = kB / int(sizeof(T));   // k of a step
  const int64_t step_a = A_ACROSS ? kK * p.lda : kK, step_b = B_ACROSS ? kK * p.ldb : kK;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 sum[MODE == kDw ? FM : 1];
#pragma unroll
  for (f32x4& v : sum) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const bool sums = MODE == kDw && p.db != nullptr && n0 == 0 && wn == 0;

  // the sets' first steps lie side by side
  const int first = k_all - set * kK;
  a += set * step_a;
  b += set * step_b;
  if (MODE == kDw && k_all == 0) {
    // an empty group's zeros
  } else if constexpr (DIRECT) {
    constexpr int kBytes = (BM + BN) * kB, kLoads = kBytes / 16 / THREADS;
    Direct<T, BM, A_ACROSS, THREADS, kB> da;
    Direct<T, BN, B_ACROSS, THREADS, kB> db;
    da.init(p.lda, tid);
    db.init(p.ldb, tid);
    // with more than two stages every step loads the same number of times, past
    // the end nothing but zeros
    int ahead = first;
    const auto load = [&](int stage) {
      char* t = lds + stage * kBytes;
      da.load(a, p.lda, A_ACROSS ? ahead : m_left, A_ACROSS ? m_left : ahead, t, wave);
      db.load(b, p.ldb, B_ACROSS ? ahead : n_left, B_ACROSS ? n_left : ahead, t + BM * kB, wave);
      ahead -= KW * kK;
      a += KW * step_a;
      b += KW * step_b;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(s);
    int stage = 0;
    for (int all = k_all, left = first; all > 0; all -= KW * kK, left -= KW * kK) {
      tile_barrier<WM * WN, (kStages - 2) * kLoads>();
      // two stages wait for everything anyway, and a single step has but one
      if (kStages > 2 || all > KW * kK) load(stage == 0 ? kStages - 1 : stage - 1);
      const char* t = lds + stage * kBytes;
      if (KW == 1 || left > 0)
        multiply_step<T, BM, BN, A_ACROSS, B_ACROSS, kB>(t, t + BM * kB, wm * TM, wn * TN, lane, acc, sum, sums);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    tile_barrier<WM * WN * KW>();
  } else {
    char* const ta = lds;
    char* const tb = lds + BM * 128;
    // rows of memory from the corners on: the weights' groups follow each other
    const int a_mem = p.rows - s.row0 - (A_ACROSS ? set * kStep<T> : 0);
    const int64_t w_rows = int64_t(std::max(1, p.groups) - s.e) * (MODE == kFwd ? p.n : p.k);
    const int64_t b_rows = MODE == kDw ? a_mem : w_rows - (MODE == kFwd ? n0 : set * kStep<T>);
    const int b_mem = b_rows < (1 << 30) ? int(b_rows) : 1 << 30;
    const bool a_narrow = (A_ACROSS ? p.m : p.k) < 8, b_narrow = (B_ACROSS ? p.n : p.k) < 8;
    Stage<T, BM, A_ACROSS, THREADS> sa;
    Stage<T, BN, B_ACROSS, THREADS> sb;
    if (KW == 1 || first > 0) {
      sa.load(a, p.lda, A_ACROSS ? first : m_left, A_ACROSS ? m_left : first, a_mem, a_narrow, tid);
      sb.load(b, p.ldb, B_ACROSS ? first : n_left, B_ACROSS ? n_left : first, b_mem, b_narrow, tid);
    }
    for (int all = k_all, left = first, done = 0; all > 0; all -= KW * kStep<T>, left -= KW * kStep<T>) {
      if (KW == 1 || left > 0) {
        sa.store(ta, tid);
        sb.store(tb, tid);
      }
      stage_barrier<WM * WN>();
      const int next = left - KW * kStep<T>;
      if (next > 0) {   // the next step's loads fly while this one is multiplied
        a += KW * step_a;
        b += KW * step_b;
        done += KW * kStep<T>;
        sa.load(a, p.lda, A_ACROSS ? next : m_left, A_ACROSS ? m_left : next, A_ACROSS ? a_mem - done : a_mem, a_narrow,
                tid);
        sb.load(b, p.ldb, B_ACROSS ? next : n_left, B_ACROSS ? n_left : next, B_ACROSS ? b_mem - done : b_mem, b_narrow,
                tid);
      }
      if (KW == 1 || left > 0)
        multiply_step<T, BM, BN, A_ACROSS, B_ACROSS, 128>(ta, tb, wm * TM, wn * TN, lane, acc, sum, sums);
      stage_barrier<WM * WN>();
    }
    if (WM * WN == 1) __syncthreads();
  }

  if constexpr (KW > 1) {
    // sets 1 .. KW - 1 leave their results in LDS, register by register
    constexpr int kRegs = FM * FN + (MODE == kDw ? FM : 0);
    f32x4* box = reinterpret_cast<f32x4*>(base);
    if (set > 0) {
      f32x4* mine = box + (set - 1) * kRegs * THREADS + tid;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mine[(i * FN + j) * THREADS] = acc[i][j];
      if constexpr (MODE == kDw)
#pragma unroll
        for (int i = 0; i < FM; ++i) mine[(FM * FN + i) * THREADS] = sum[i];
    }
    __syncthreads();
    if (set > 0) return;
#pragma unroll
    for (int q = 0; q < KW - 1; ++q) {
      const f32x4* theirs = box + q * kRegs * THREADS + tid;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] += theirs[(i * FN + j) * THREADS];
      if constexpr (MODE == kDw)
#pragma unroll
        for (int i = 0; i < FM; ++i) sum[i] += theirs[(FM * FN + i) * THREADS];
    }
    lds = base + (KW - 1) * kRegs * THREADS * 16;   // the patches lie past the boxes, which others may still read
  }

  // Epilogue: 16 rows at a time through the wave's patch.  A lane has the
  // same eight columns in every pass, so their bias stays in registers; the
  // residual's chunks are all asked for before the first is needed.
  constexpr int kAcross = TN / 8, kRows = 64 / kAcross, kPasses = 16 / kRows;   // lanes of a row, rows a pass
  constexpr int kBatch = std::min(FM, (FM > 4 ? 8 : 16) / (kPasses * Eight<T>::kParts));   // their residual in flight
  const int col = wn * TN + (lane % kAcross) * 8, n = std::min(8, n_left - col);
  const int64_t row0 = MODE == kDw ? m0 : s.row0;
  float* plane = nullptr;
  void* out = p.out;
  if constexpr (MODE == kDw) {
    if (p.part != nullptr && s.slots > 1)
      plane = p.part + int64_t(stretch) * p.plane;
    else
      out = p.out_f32 ? static_cast<void*>(static_cast<float*>(p.out) + int64_t(s.e) * p.m * p.ldo)
                      : static_cast<void*>(static_cast<T*>(p.out) + int64_t(s.e) * p.m * p.ldo);
  }
  if constexpr (MODE == kDw) {
    if (sums && lane < 16) {   // lane m has the sum of column m in every register
      float* o = plane != nullptr ? plane + int64_t(p.m) * p.n : p.db + int64_t(s.e) * p.m;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = wm * TM + 16 * i + lane;
        if (m < m_left) o[m0 + m] = sum[i][0];
      }
    }
    if (p.out == nullptr) return;   // no rows and db alone: its zeros
  }
  float bias[8];
  if constexpr (MODE == kFwd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = p.bias != nullptr && i < n ? p.bias[int64_t(s.e) * p.n + n0 + col + i] : 0.0f;
  }
  float* patch = reinterpret_cast<float*>(lds) + wave * 16 * kPatch;
#pragma unroll
  for (int i0 = 0; i0 < FM; i0 += kBatch) {
    Eight<T> res[kBatch * kPasses];
    if (MODE == kFwd && p.residual != nullptr) {
#pragma unroll
      for (int q = 0; q < kBatch * kPasses; ++q) {
        const int m = wm * TM + 16 * (i0 + q / kPasses) + (q % kPasses) * kRows + lane / kAcross;
        res[q].load(static_cast<const T*>(p.residual) + (row0 + m) * p.ldr + n0 + col, m < m_left ? n : 0);
      }
    }
#pragma unroll
    for (int i = i0; i < i0 + kBatch; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f32x4*>(patch + (lane & 15) * kPatch + 16 * j + 4 * (lane >> 4)) = acc[i][j];
      wave_sync();
#pragma unroll
      for (int q = 0; q < kPasses; ++q) {
        const int r = q * kRows + lane / kAcross, m = wm * TM + 16 * i + r;
        float v[8];
        const f32x4 lo = *reinterpret_cast<const f32x4*>(patch + r * kPatch + (lane % kAcross) * 8);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(patch + r * kPatch + (lane % kAcross) * 8 + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[c] = lo[c];
          v[4 + c] = hi[c];
        }
        if (m >= m_left || n <= 0) continue;
        const int64_t row = row0 + m;
        if (MODE == kDw && (plane != nullptr || p.out_f32)) {
          Eight<float> o;
          o.set(v);
          o.store(plane != nullptr ? plane + row * p.n + n0 + col : static_cast<float*>(out) + row * p.ldo + n0 + col,
                  n);
          continue;
        }
        Eight<T> o;
        if constexpr (MODE == kFwd) {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] += bias[c];
          if (p.z != nullptr) {
            o.set(v);
            o.store(static_cast<T*>(p.z) + row * p.ldz + n0 + col, n);
          }
          act_eight<T>(v, p.act);
          if (p.residual != nullptr) {
            const Eight<T>& x = res[(i - i0) * kPasses + q];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] += x.get(c);
          }
        }
        o.set(v);
        o.store(static_cast<T*>(out) + row * p.ldo + n0 + col, n);
      }
      wave_sync();
    }
  }
}

// LDS of a workgroup: the stages of its sets (256 bytes of k in all of them
// together; one step of 128 where the tiles come through registers or there
// is but one), later the boxes of the sets' results and the patches.
constexpr int product_lds(int bm, int bn, int wm, int wn, int kw, bool staged) {
  const int tiles = (bm + bn) * (staged ? 256 : 128) * kw;
  const int regs = (bm / wm / 16) * (bn / wn / 16 + 1);   // kDw's, the largest
  const int after = (kw - 1) * regs * 64 * wm * wn * 16 + wm * wn * 16 * (bn / wn + 4) * 4;
  return tiles > after ? tiles : after;
}

// Workgroup `id` of `grid` of a product.
template <typename T, Mode MODE, int BM, int BN, int WM, int WN, bool DIRECT, int KW>
__device__ __forceinline__ void product_block(const ProductArgs& p, int id, int grid, char* lds) {
  // the grid is sized for the most slots the groups can make; the tiles that
  // there are go evenly to the XCDs
  int tiles = grid;
  if (p.groups > 0 && (MODE != kDw || p.part != nullptr)) {
    tiles = total_slots(p.offsets, p.groups, p.rows, p.unit) * (MODE == kDw ? p.tiles : p.tiles_n);
    if (id >= tiles) return;
  }
  int tile = xcd_tile(id, tiles);
  if (MODE != kDw && p.tiles_n >= 8) {
    // kRun heights at a time, all their tiles across: what runs together on an
    // XCD shares rows and weights about evenly (16384 x 4096 x 4096 fp16: 490 ->
    // 470 us; below 8 tiles across the heights are as near anyway)
    constexpr int kRun = 4;
    const int run = tile / (kRun * p.tiles_n), in = tile - run * kRun * p.tiles_n;
    const int high = std::min(kRun, tiles / p.tiles_n - run * kRun);
    tile = (run * kRun + in % high) * p.tiles_n + in / high;
  }
  product_tile<T, MODE, BM, BN, WM, WN, DIRECT, KW>(p, tile, lds);
}

template <typename T, Mode MODE, int BM, int BN, int WM, int WN, bool DIRECT, int KW>
__global__ __launch_bounds__(64 * WM * WN * KW, KW == 4 ? 4 : 2) void k_product(ProductArgs p) {
  extern __shared__ __align__(16) char lds[];
  product_block<T, MODE, BM, BN, WM, WN, DIRECT, KW>(p, blockIdx.x, gridDim.x, lds);
}

// dw and dx of ragged groups, both in 256 x 256 tiles, a workgroup a CU: dw's
// workgroups last as long as their groups, so dx's, short and alike, fill the
// CUs that the smaller groups leave.  The whole backward in bf16 with silu against
// two launches: 131,072 rows on 64 ragged heads 512 -> 512 328 us, 368; 262,144 on
// 16 649 us, 766; 100,000 on 32 768 -> 512 327 us, 414.  (Without groups the two
// are within 4 % of each other, either way.)
template <typename T>
__global__ __launch_bounds__(512, 2) void k_bwd_groups(ProductArgs x, ProductArgs w, int w_grid) {
  extern __shared__ __align__(16) char lds[];
  const int b = blockIdx.x;
  if (b < w_grid)
    product_block<T, kDw, 256, 256, 2, 4, true, 1>(w, b, w_grid, lds);
  else
    product_block<T, kDx, 256, 256, 2, 4, true, 1>(x, b - w_grid, int(gridDim.x) - w_grid, lds);
}

// --- the product over many rows of a short k ---------------------------------------

// For k of at most four steps: the weights are a constant of the kernel, not
// an operand to stream.  Each of 8 waves keeps the fragments of its 32 output
// columns in registers (KS * 16 of them) and the workgroup walks its share of
// the row tiles, 16 KB of rows a tile, three LDS stages deep, so that rows are
// read from HBM once and loads are always in flight.  Every tile issues the
// same number of memory instructions (buffer loads and stores, whose rows
// past the end are dropped by the buffer's size), which lets the wait for a
// stage count them instead of draining the stores of the tile before.
// 128 / KS rows a tile, WM x WN = 8 waves of 128 / KS / WM x 32 outputs.
// Bound by HBM: 1,000,000 rows, bf16: 256 -> 256 213 us, 4.8 TB/s (340 us with
// 128 x 128 tiles, whose loads stop for the epilogue); 64 -> 256 with gelu
// and z 270 us, 4.3 TB/s (324 us).

template <int N>
__device__ __forceinline__ void rows_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N < 63 ? N : 63) : "memory");   // the counter holds 6 bits
}

#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the buffer builtins
// A wave-uniform address range for buffer instructions.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(T* p, int64_t ld, int rows, int cols) {
  const uint32_t bytes = rows > 0 ? uint32_t(((rows - 1) * ld + cols) * int64_t(sizeof(T))) : 0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<std::remove_const_t<T>*>(p), 0, bytes, 0x00020000);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ void buffer_store_eight(__amdgpu_buffer_rsrc_t r, const Eight<T>& e, uint32_t off) {
#pragma unroll
  for (int h = 0; h < Eight<T>::kParts; ++h)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, e.c[h]), r, off + 16u * h, 0, 0);
}
template <typename T>
__device__ __forceinline__ void buffer_load_eight(__amdgpu_buffer_rsrc_t r, Eight<T>& e, uint32_t off) {
#pragma unroll
  for (int h = 0; h < Eight<T>::kParts; ++h)
    e.c[h] = __builtin_bit_cast(Chunk<T>, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16u * h, 0, 0));
}
#endif

template <typename T, Mode MODE, int KS, int WM, int WN>
__global__ __launch_bounds__(512, 4) void k_rows(ProductArgs p, int shares) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int BM = 128 / KS, TM = BM / WM, FM = TM / 16, FB = std::min(FM, 4), FN = 2, BN = WN * 32;
  static_assert(WM * WN == 8 && TM >= 16, "8 waves of 32 columns");
  constexpr int kStage = 16384, kStages = 3, kPatch = 36;
  constexpr int kLoads = 2;                                  // loads of a stage a thread: 1024 chunks over 512
  constexpr int kPlane = FM * Eight<T>::kParts;              // memory instructions of one output or residual plane
  __shared__ __align__(16) char lds[kStages * kStage + 8 * 16 * kPatch * 4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  float* patch = reinterpret_cast<float*>(lds + kStages * kStage) + wave * 16 * kPatch;

  // the share of row tiles and the column tile
  const int id = xcd_tile(blockIdx.x, gridDim.x), n0 = id % p.tiles_n * BN, share = id / p.tiles_n;
  const int64_t total = total_slots(p.offsets, p.groups, p.rows, BM);
  const int t0 = int(total * share / shares), t1 = int(total * (share + 1) / shares);
  if (t0 >= t1) return;
  const int n_left = p.n - n0;

  // chunk this thread fetches: 8 chunks of a row and step, row by row, step by step
  uint32_t off[kLoads];
  bool in_k[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int at = j * 512 + tid, step = at / (BM * 8), r = at / 8 % BM, c = (at & 7) ^ (r & 7);
    off[j] = uint32_t(r) * uint32_t(p.lda * sizeof(T)) + uint32_t(step * 128 + c * 16);
    in_k[j] = (step * 8 + c) * kChunk<T> < p.k;
    if (!in_k[j]) off[j] = 0xfffffff0u;
  }
  const auto fetch = [&](const Span& s, int stage) {
    const __amdgpu_buffer_rsrc_t r = buffer_of(static_cast<const T*>(p.a) + int64_t(s.row0) * p.lda, p.lda,
                                               s.e < 0 ? 0 : s.row1 - s.row0, p.k);
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void*)(lds + stage * kStage + j * 8192 + wave * 1024), 16, off[j], 0, 0,
          0);
  };

  // the tile after `s`, inside its group or in the next one
  const auto after = [&](const Span& s, int t) {
    if (t >= t1) return Span{-1, 0, 0, 0, 0, 0};
    if (p.groups > 0 && t >= s.slot0 + s.slots) return find_span(p.offsets, p.groups, p.rows, BM, t);
    Span q = s;
    q.row0 = s.row0 + BM;
    q.row1 = s.end - q.row0 < BM ? s.end : q.row0 + BM;
    return q;
  };
  Span now = find_span(p.offsets, p.groups, p.rows, BM, t0), next = after(now, t0 + 1);
  fetch(now, 0);
  fetch(next, 1);

  typename Frag<T>::V fw[KS * 2][FN];
  float bias[8];
  const int col = wn * 32 + (lane & 3) * 8;                  // of this lane in the epilogue
  const bool live = col < n_left;                            // n_left is whole chunks of 8
  int group = -1, stage = 0;
  const int planes = 1 + (p.z != nullptr) + (p.residual != nullptr);

  for (int t = t0; t < t1; ++t) {
    // after this stage's loads come: the next stage's, and the last two
    // tiles' epilogues (less of both at the start)
    if (t - t0 < 2)
      rows_barrier<kLoads>();
    else if (planes == 1)
      rows_barrier<kLoads + 2 * kPlane>();
    else if (planes == 2)
      rows_barrier<kLoads + 4 * kPlane>();
    else
      rows_barrier<kLoads + 6 * kPlane>();
    const Span later = after(next, t + 2);
    fetch(later, stage == 0 ? 2 : stage - 1);
    asm volatile("" ::: "memory");   // the counted order: these loads, then the epilogue

    if (now.e != group) {
      group = now.e;
      const T* w = static_cast<const T*>(p.b) + int64_t(group) * p.b_group;
      int ln = lane;
      asm volatile("" : "+v"(ln));   // addresses are made here, not kept through the loop
#pragma unroll
      for (int kk = 0; kk < KS * 2; ++kk)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int n = n0 + wn * 32 + 16 * j + (ln & 15), k = (4 * kk + (ln >> 4)) * kChunk<T>;
          Chunk<T> c;
          if constexpr (MODE == kFwd) {   // k is whole chunks: all of one or none
            c = load_chunk(w + int64_t(std::min(n, p.n - 1)) * p.ldb + (k < p.k ? k : 0));
#pragma unroll
            for (int i = 0; i < kChunk<T>; ++i) c.v[i] = n < p.n && k < p.k ? c.v[i] : T(0.0f);
          } else {
            const T* q = w + std::min(n, p.n - 1) + int64_t(k < p.k ? k : 0) * p.ldb;
#pragma unroll
            for (int i = 0; i < kChunk<T>; ++i) c.v[i] = q[i * p.ldb];
#pragma unroll
            for (int i = 0; i < kChunk<T>; ++i) c.v[i] = n < p.n && k < p.k ? c.v[i] : T(0.0f);
          }
          fw[kk][j] = __builtin_bit_cast(typename Frag<T>::V, c);
          if (MODE == kDx) __builtin_amdgcn_sched_barrier(0);   // a fragment's values at a time: no spills
        }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        bias[i] = MODE == kFwd && p.bias != nullptr && live ? p.bias[int64_t(group) * p.n + n0 + col + i] : 0.0f;
    }

    const int rows = now.row1 - now.row0, m0 = wm * TM + (lane >> 2);
    const bool add = MODE == kFwd && p.residual != nullptr;
    const auto rr = buffer_of(static_cast<const T*>(p.residual) + int64_t(now.row0) * p.ldr + n0, p.ldr, rows, n_left);
    const auto ro = buffer_of(static_cast<T*>(p.out) + int64_t(now.row0) * p.ldo + n0, p.ldo, rows, n_left);
    const auto rz = buffer_of(static_cast<T*>(p.z) + int64_t(now.row0) * p.ldz + n0, p.ldz, rows, n_left);
    const auto at = [&](int i, int64_t ld) {   // byte offset of this lane's eight values in rows 16 i ..
      return live ? uint32_t(m0 + 16 * i) * uint32_t(ld * sizeof(T)) + uint32_t(col * sizeof(T)) : 0xffffff00u;
    };
    const char* tile = lds + stage * kStage;
    Eight<T> res;
    if (add) buffer_load_eight(rr, res, at(0, p.ldr));
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += FB) {
      f32x4 acc[FB][FN];
#pragma unroll
      for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KS * 2; ++kk) {
        typename Frag<T>::V fa[FB];
#pragma unroll
        for (int i = 0; i < FB; ++i)
          fa[i] = read_frag<T, BM, false>(tile + (kk >> 1) * BM * 128, wm * TM + 16 * (i0 + i), kk & 1, lane);
        mma_all<T, FB, FN>(fw[kk], fa, acc);
      }
#pragma unroll
      for (int i = 0; i < FB; ++i) {
        Eight<T> ahead;
        if (add && i0 + i + 1 < FM) buffer_load_eight(rr, ahead, at(i0 + i + 1, p.ldr));
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4*>(patch + (lane & 15) * kPatch + 16 * j + 4 * (lane >> 4)) = acc[i][j];
        wave_sync();
        const f32x4 lo = *reinterpret_cast<const f32x4*>(patch + (lane >> 2) * kPatch + (lane & 3) * 8);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(patch + (lane >> 2) * kPatch + (lane & 3) * 8 + 4);
        float v[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[c] = lo[c];
          v[4 + c] = hi[c];
        }
        Eight<T> o;
        if constexpr (MODE == kFwd) {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] += bias[c];
          if (p.z != nullptr) {
            o.set(v);
            buffer_store_eight(rz, o, at(i0 + i, p.ldz));
          }
          act_eight<T>(v, p.act);
          if (add) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] += res.get(c);
            res = ahead;
          }
        }
        o.set(v);
        buffer_store_eight(ro, o, at(i0 + i, p.ldo));
        wave_sync();
      }
    }
    now = next;
    next = later;
    stage = stage == 2 ? 0 : stage + 1;
  }
  rows_barrier<0>();   // no load into LDS outlives the workgroup
#endif
}

// --- dz and db ----------------------------------------------------------------------------------

// dz = dy act'(z) rounded into the storage type, and one partial row of db per
// stretch of rows, part[slot][out], or without `part` db itself, one stretch a
// group.  The rounding is a choice: one matrix instruction takes 16-bit values,
// and a dz of a high and a low part would double both products' instructions
// and LDS reads and the bytes of dz; dx and dw then have 1.4 times the error of a 32-bit
// dz (1,000,000 x 256 -> 256 bf16: 0.0024 of their norm against 0.0017), as a
// program of 16-bit tensors has.  db is summed from the unrounded values, in
// fp32.  No dz: the sums of dy alone.
template <typename T>
__global__ __launch_bounds__(256) void k_act_grad(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ z,
                                                  int64_t ldz, T* __restrict__ dz, int64_t lddz,
                                                  const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                                  int32_t unit, int32_t out, int act, int lanes,
                                                  float* __restrict__ part, float* __restrict__ db) {
  constexpr int K = kChunk<T>;
  __shared__ float s[256][K + 1];
  const Span sp = part == nullptr ? group_span(offsets, groups, rows, unit, blockIdx.x)
                                  : find_span(offsets, groups, rows, unit, blockIdx.x);
  if (sp.e < 0) return;
  const int cl = threadIdx.x % lanes, rl = threadIdx.x / lanes, col = (blockIdx.y * lanes + cl) * K;
  const int n = std::min(K, std::max(0, out - col));
  float sum[K];
#pragma unroll
  for (int i = 0; i < K; ++i) sum[i] = 0.0f;
  if (n > 0)
#pragma unroll 4
    for (int64_t r = sp.row0 + rl; r < sp.row1; r += 256 / lanes) {
      const Chunk<T> c = load_chunk_n(dy + r * lddy + col, n);
      float v[K];
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = float(c.v[i]);
      if (dz != nullptr) {
        const Chunk<T> zc = load_chunk_n(z + r * ldz + col, n);
        Chunk<T> o;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          v[i] *= act_slope<T>(float(zc.v[i]), act);
          o.v[i] = T(v[i]);
        }
        store_chunk(dz + r * lddz + col, o);   // lddz is whole chunks: the padding is written too
      }
#pragma unroll
      for (int i = 0; i < K; ++i) sum[i] += v[i];
    }
  float* __restrict__ to = part != nullptr ? part + int64_t(blockIdx.x) * out : db != nullptr ? db + int64_t(sp.e) * out
                                                                                            : nullptr;
  if (to == nullptr) return;
#pragma unroll
  for (int i = 0; i < K; ++i) s[threadIdx.x][i] = sum[i];
  __syncthreads();
  for (int step = 128; step >= lanes; step >>= 1) {
    if (int(threadIdx.x) < step)
#pragma unroll
      for (int i = 0; i < K; ++i) s[threadIdx.x][i] += s[threadIdx.x + step][i];
    __syncthreads();
  }
  if (rl == 0)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (i < n) to[col + i] = s[threadIdx.x][i];
}

// Joins planes that lie `plane` apart, n of them from q on: values are shared
// out 64 a workgroup, their planes among its four waves, whose sums are added
// in order.
__device__ __forceinline__ float join_planes(const float* __restrict__ q, int64_t plane, int n, bool live,
                                             float (&box)[256]) {
  const int w = threadIdx.x >> 6;
  float v = 0.0f;
  if (live)
#pragma unroll 8
    for (int t = w; t < n; t += 4) v += q[t * plane];
  if (n > 1) {
    __syncthreads();   // the box's last readers
    box[threadIdx.x] = v;
    __syncthreads();
    if (w == 0) v = (box[threadIdx.x] + box[threadIdx.x + 64]) + (box[threadIdx.x + 128] + box[threadIdx.x + 192]);
  }
  return v;
}

// Joins the planes of dw (size values, then m of db).  Groups of one
// stretch were written by the product itself; empty ones are 0.
template <typename O>
__global__ __launch_bounds__(256) void k_join(const float* __restrict__ part, int64_t plane,
                                              const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                              int32_t unit, int64_t size, O* __restrict__ out, int32_t m,
                                              float* __restrict__ db) {
  __shared__ float box[256];
  const Span s = group_span(offsets, groups, rows, unit, blockIdx.y);
  if (s.slots == 1) return;
  const int64_t all = size + (db != nullptr ? m : 0);
  for (int64_t i0 = int64_t(blockIdx.x) * 64; i0 < all; i0 += int64_t(gridDim.x) * 64) {
    const int64_t i = i0 + (threadIdx.x & 63);
    const float v = join_planes(part + int64_t(s.slot0) * plane + i, plane, s.slots, i < all, box);
    if (threadIdx.x >= 64 || i >= all) continue;
    if (i < size)
      out[int64_t(blockIdx.y) * size + i] = O(v);
    else
      db[int64_t(blockIdx.y) * m + (i - size)] = v;
  }
}

// db from the partial rows of k_act_grad: `cols` columns a workgroup, 256 /
// cols shares of a group's rows, joined in a fixed order.
struct DbJoin {
  const float* part;
  float* db;
  int32_t out, unit, cols, blocks;   // blocks: workgroups of a group
};
__device__ __forceinline__ void join_db(const DbJoin& j, const ProductArgs& p, int block, float* box) {
  const Span s = group_span(p.offsets, p.groups, p.rows, j.unit, block / j.blocks);
  const int tid = threadIdx.x, c = tid % j.cols, share = tid / j.cols, shares = 256 / j.cols;
  const int col = block % j.blocks * j.cols + c;
  if (tid < 256) {
    float v = 0.0f;
    if (col < j.out)
#pragma unroll 4
      for (int t = share; t < s.slots; t += shares) v += j.part[(int64_t(s.slot0) + t) * j.out + col];
    box[tid] = v;
  }
  __syncthreads();
  if (tid >= j.cols || col >= j.out) return;
  float v = 0.0f;
  for (int t = 0; t < shares; ++t) v += box[j.cols * t + tid];
  j.db[int64_t(s.e) * j.out + col] = v;
}
__global__ __launch_bounds__(256) void k_join_db(DbJoin j, ProductArgs p) {
  __shared__ float box[256];
  join_db(j, p, blockIdx.x, box);
}

// Small problems, whose cost is their launches: dx, dw and what is left of
// db in one, the workgroups shared out among the three.  Tiles of 64 x 64, or
// of 32 x 32 with eight wave sets where the k of one of them is long.
template <typename T, int TILE, int W, bool DIRECT, int KW>
__global__ __launch_bounds__(64 * W * W * KW) void k_bwd(ProductArgs x, int x_tiles, ProductArgs w, int w_tiles, DbJoin j) {
  extern __shared__ __align__(16) char lds[];
  // dw's workgroups, the longest, first (50,001 rows 251 -> 59 fp32, the whole
  // backward: 69 us, 86 us with them last)
  int b = blockIdx.x;
  if (b < w_tiles) {
    product_tile<T, kDw, TILE, TILE, W, W, DIRECT, KW>(w, b, lds);
    return;
  }
  b -= w_tiles;
  if (b < x_tiles)
    product_tile<T, kDx, TILE, TILE, W, W, DIRECT, KW>(x, b, lds);
  else
    join_db(j, w, b - x_tiles, reinterpret_cast<float*>(lds));
}

// --- the whole backward pass over many rows of a narrow layer --------------------------

struct FusedArgs {
  const void* dy;
  const void* z;       // NULL: no activation
  const void* x;
  const void* w;
  void* dx;            // or NULL, and w with it
  float* part;         // planes of [m = out][n = in], then [m] of db
  const int64_t* offsets;
  int64_t lddy, ldz, ldx, ldw, lddx, w_group, plane;
  int32_t rows, groups, in, out, act;
  int32_t shares;      // at most
};

// The tiles lie in the rows that groups cover, which may be few of them: no
// more shares than tiles, so that every share has a tile and writes its planes
// (k_join_rows adds all planes between a group's first share and its last).
__device__ __forceinline__ int32_t shares_in_use(int64_t total, int32_t shares) {
  return total < shares ? int32_t(total) : shares;
}

// Which share of the tiles tile t is in: share s holds total s / shares ..
// total (s + 1) / shares - 1.
__host__ __device__ inline int32_t share_of(int64_t t, int64_t total, int32_t shares) {
  int64_t s = t * shares / total;
  while (total * (s + 1) / shares <= t) ++s;
  return int32_t(s);
}

// Layers of up to 64 KO columns out and 64 KI in (KO, KI = 1, 2, 4): one pass
// reads dy, z and x and writes dx, and dw never leaves the registers until the
// rows run out.  Each of 8 waves holds the weights' fragments of 32 columns of
// dx (16 KO registers) and an eighth of dw's sums (up to 128); the workgroup
// walks its share of the row tiles (128 / max(KO, KI) rows; dy, z, x up to 16 KB
// each, two tiles in flight with counted waits):
//   slope   dz = dy act'(z) in place, rounded into the storage type (as in
//           k_act_grad), db summed unrounded
//   product dx = dz w; dw += dz^T x, its operands read transposed
// A share that ends inside a group, or a group inside a share, leaves one
// plane of partial sums, number share + group.  What it has to move is 3 or 4
// planes of the rows, each once; what bounds it at 256 x 256 is the issue of
// one tile's phases one after the other on 2 waves a SIMD (the vector unit is
// busy half of the time, the matrix unit a fifth): 1,000,000 rows with gelu 583
// us, 3.5 TB/s, where a pass for dz and two products took 972 us.  Measured
// and not taken: slopes a tile ahead in turn with the products of the other
// wave of a SIMD (645 us), x fetched a tile further ahead (no change).
template <typename T, int KO, int KI>
__global__ __launch_bounds__(512, 2) void k_bwd_rows(FusedArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  static_assert(sizeof(T) == 2, "transposed LDS reads are 16 bit");
  constexpr int BM = 128 / std::max(KO, KI), K = 8, FN = 2;
  // dx: WM x WN waves of TM x 32 outputs (of the narrowest, some have none)
  constexpr int WN = 2 * KI, WM = std::min(8 / WN, BM / 16), TM = BM / WM, FM = TM / 16;
  // dw: WO x WI waves
  constexpr int WO = KO == KI ? 4 : KO == 4 * KI ? 8 : KO > KI ? 4 : KI == 4 * KO ? 1 : 2, WI = 8 / WO;
  constexpr int DM = KO * 4 / WO, DN = KI * 4 / WI;
  constexpr int kPatch = 40, kStores = FM * Eight<T>::kParts;
  // tiles in LDS: of whole kilobytes for every wave, so that each has as many loads
  constexpr int kLoadsY = (BM * KO * 128 + 8191) / 8192, kLoadsX = (BM * KI * 128 + 8191) / 8192;
  constexpr int kTileY = kLoadsY * 8192, kTileX = kLoadsX * 8192;
  // three tiles each of dy (then dz), x and z, the patches (in the storage
  // type: nothing is added to dx), and 16 KB for db's sums, which lie in a z
  // tile where that is large enough
  constexpr int kPatches = 8 * 16 * kPatch * 2;
  constexpr bool kBoxInZ = kTileY >= 16384;
  __shared__ __align__(16) char lds[6 * kTileY + 3 * kTileX + kPatches + (kBoxInZ ? 0 : 16384)];
  char* const lds_z = lds + 3 * kTileY;
  char* const lds_x = lds + 6 * kTileY;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  const bool has_dx = p.dx != nullptr && wm < WM;
  T* patch = reinterpret_cast<T*>(lds_x + 3 * kTileX) + wave * 16 * kPatch;

  const int64_t total = total_slots(p.offsets, p.groups, p.rows, BM);
  const int shares = shares_in_use(total, p.shares);
  const int share = xcd_tile(blockIdx.x, gridDim.x);
  if (share >= shares) return;
  const int t0 = int(total * share / shares), t1 = int(total * (share + 1) / shares);

  // a thread's chunks of a tile: 8 of a row and step, row by row, step by step
  const auto fetch_one = [&](auto loads, auto steps, const void* q, int64_t ld, int cols, const Span& s, int th,
                             char* to) {
    const __amdgpu_buffer_rsrc_t rsrc =
        buffer_of(static_cast<const T*>(q) + int64_t(s.row0) * ld, ld, s.e < 0 ? 0 : s.row1 - s.row0, cols);
#pragma unroll
    for (int j = 0; j < decltype(loads)::value; ++j) {
      const int at = j * 512 + th, step = at / (BM * 8), r = at / 8 % BM, col = (step * 8 + ((at & 7) ^ (r & 7))) * K;
      const uint32_t off = col < cols && step < decltype(steps)::value ? __umul24(r, uint32_t(ld * 2)) + uint32_t(col * 2) : 0xfffffff0u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(to + j * 8192 + wave * 1024), 16, off, 0, 0, 0);
    }
  };
  const auto fetch = [&](const Span& s, int ring) {
    int th = tid;
    asm volatile("" : "+v"(th));   // addresses kept through the loop would spill
    using std::integral_constant;
    const integral_constant<int, kLoadsY> ly{};
    const integral_constant<int, kLoadsX> lx{};
    const integral_constant<int, KO> ko{};
    const integral_constant<int, KI> ki{};
    fetch_one(ly, ko, p.dy, p.lddy, p.out, s, th, lds + ring * kTileY);
    if (p.z != nullptr) fetch_one(ly, ko, p.z, p.ldz, p.out, s, th, lds_z + ring * kTileY);
    fetch_one(lx, ki, p.x, p.ldx, p.in, s, th, lds_x + ring * kTileX);
  };
  const auto after = [&](const Span& s, int t) {
    if (t >= t1) return Span{-1, 0, 0, 0, 0, 0};
    if (p.groups > 0 && t >= s.slot0 + s.slots) return find_span(p.offsets, p.groups, p.rows, BM, t);
    Span q = s;
    q.row0 = s.row0 + BM;
    q.row1 = s.end - q.row0 < BM ? s.end : q.row0 + BM;
    return q;
  };
  Span now = find_span(p.offsets, p.groups, p.rows, BM, t0), next = after(now, t0 + 1);
  fetch(now, 0);
  fetch(next, 1);

  typename Frag<T>::V fw[KO * 2][FN];
  f32x4 dw[DM][DN];
  float db[K];
#pragma unroll
  for (int i = 0; i < DM; ++i)
#pragma unroll
    for (int j = 0; j < DN; ++j) dw[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < K; ++i) db[i] = 0.0f;
  // dz: a thread's chunk column is the same in all its rows
  constexpr int kCols = KO * 8, kApart = 512 / kCols;    // chunk columns, rows between a thread's rows
  const int am = wave / WI * 16 * DM, bn = wave % WI * 16 * DN;   // this wave's corner of dw
  Across across_y, across_x;   // of its blocks, which may begin inside a step
  across_y.init(lane, (am >> 4) & 3);
  across_x.init(lane, (bn >> 4) & 3);
  const auto slope = [&](int ring) {
    char* const ty = lds + ring * kTileY;
    const char* const tz = lds_z + ring * kTileY;
    int th = tid;
    asm volatile("" : "+v"(th));
    const int zc = th % kCols, zr = th / kCols;
#pragma unroll
    for (int j = 0; j < (BM + kApart - 1) / kApart; ++j) {
      const int r = zr + j * kApart;
      if (BM < kApart && r >= BM) break;
      const int at = (zc >> 3) * BM * 128 + tile_at<T, BM, false>(r, zc & 7);
      Chunk<T> c = *reinterpret_cast<const Chunk<T>*>(ty + at);
      if (p.z != nullptr) {
        const Chunk<T> q = *reinterpret_cast<const Chunk<T>*>(tz + at);
        float s[8];
#pragma unroll
        for (int i = 0; i < K; ++i) s[i] = float(q.v[i]);
        slope_eight<T>(s, p.act);
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const float v = float(c.v[i]) * s[i];
          db[i] += v;
          c.v[i] = T(v);
        }
        *reinterpret_cast<Chunk<T>*>(ty + at) = c;
      } else {
#pragma unroll
        for (int i = 0; i < K; ++i) db[i] += float(c.v[i]);
      }
    }
  };

  int group = -1, ring = 0;
  for (int t = t0; t < t1; ++t) {
    // behind this tile's loads lie the next one's and two tiles' stores (less
    // of them at the start)
    constexpr int kFetch = kLoadsY + kLoadsX;
    if (p.z == nullptr) {
      if (t - t0 < 2 || !has_dx)
        rows_barrier<kFetch>();
      else
        rows_barrier<kFetch + 2 * kStores>();
    } else {
      if (t - t0 < 2 || !has_dx)
        rows_barrier<kFetch + kLoadsY>();
      else
        rows_barrier<kFetch + kLoadsY + 2 * kStores>();
    }
    const Span later = after(next, t + 2);
    const int ring1 = ring == 2 ? 0 : ring + 1, ring2 = ring1 == 2 ? 0 : ring1 + 1;
    fetch(later, ring2);
    asm volatile("" ::: "memory");
    slope(ring);

    if (next.e != now.e) {
      // the group or the share ends with tile t: a column's sums of db lie
      // kCols threads apart, joined where this tile's z was
      float* plane = p.part + int64_t(share + now.e) * p.plane;
      float* box = reinterpret_cast<float*>(kBoxInZ ? lds_z + ring * kTileY : lds_x + 3 * kTileX + kPatches);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < K; ++i) {
        box[i * 512 + tid] = db[i];
        db[i] = 0.0f;
      }
      __syncthreads();
      if (tid < kCols * K) {
        const float* b = box + tid / kCols * 512 + tid % kCols;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kApart; ++q) v += b[q * kCols];
        const int m = (tid % kCols) * K + tid / kCols;
        if (m < p.out) plane[int64_t(p.out) * p.in + m] = v;
      }
    }

    if (now.e != group) {
      group = now.e;
      if (has_dx) {
        const T* w = static_cast<const T*>(p.w) + int64_t(group) * p.w_group;
        int ln = lane;
        asm volatile("" : "+v"(ln));
#pragma unroll
        for (int kk = 0; kk < KO * 2; ++kk)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const int n = wn * 32 + 16 * j + (ln & 15), k = (4 * kk + (ln >> 4)) * K;
            const T* q = w + std::min(n, p.in - 1) + int64_t(k < p.out ? k : 0) * p.ldw;
            Chunk<T> c;
#pragma unroll
            for (int i = 0; i < K; ++i) c.v[i] = q[i * p.ldw];
#pragma unroll
            for (int i = 0; i < K; ++i) c.v[i] = n < p.in && k < p.out ? c.v[i] : T(0.0f);
            fw[kk][j] = __builtin_bit_cast(typename Frag<T>::V, c);
            __builtin_amdgcn_sched_barrier(0);
          }
      }
    }

    if (p.z != nullptr) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const char* const ty = lds + ring * kTileY;
    const char* const tx = lds_x + ring * kTileX;
    int ln = lane;
    asm volatile("" : "+v"(ln));   // as in fetch
    if (has_dx) {
      const auto ro = buffer_of(static_cast<T*>(p.dx) + int64_t(now.row0) * p.lddx, p.lddx, now.row1 - now.row0, p.in);
      f32x4 acc[FM][FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KO * 2; ++kk) {
        typename Frag<T>::V fa[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[i] = read_frag<T, BM, false>(ty + (kk >> 1) * BM * 128, wm * TM + 16 * i, kk & 1, ln);
        mma_all<T, FM, FN>(fw[kk], fa, acc);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          struct alignas(8) Four {
            T v[4];
          } q;
#pragma unroll
          for (int c = 0; c < 4; ++c) q.v[c] = T(acc[i][j][c]);
          *reinterpret_cast<Four*>(patch + (ln & 15) * kPatch + 16 * j + 4 * (ln >> 4)) = q;
        }
        wave_sync();
        Eight<T> o;
        o.c[0] = *reinterpret_cast<const Chunk<T>*>(patch + (ln >> 2) * kPatch + (ln & 3) * 8);
        const int r = wm * TM + 16 * i + (ln >> 2), col = wn * 32 + (ln & 3) * 8;
        buffer_store_eight(ro, o, col < p.in ? __umul24(r, uint32_t(p.lddx * 2)) + uint32_t(col * 2) : 0xffffff00u);
        wave_sync();
      }
    }

    // dw: rows past the group's end are 0 in both operands.  The corners of
    // a wave's block: whole steps, but for DM = 1, 2 the columns inside one.
    const char* const wy = ty + (am >> 6) * BM * 128;
    const char* const wx = tx + (bn >> 6) * BM * 128;
#pragma unroll
    for (int kk = 0; kk < BM / 32; ++kk) {
      typename Frag<T>::V fa[DM], fb[2];
      fb[0] = across_x.template read<T, BM>(wx, 0, kk);
#pragma unroll
      for (int i = 0; i < DM; ++i) fa[i] = across_y.template read<T, BM>(wy, i, kk);
#pragma unroll
      for (int j = 0; j < DN; ++j) {   // the next fragment is read while this one is multiplied
        if (j + 1 < DN) fb[(j + 1) & 1] = across_x.template read<T, BM>(wx, j + 1, kk);
#pragma unroll
        for (int i = 0; i < DM; ++i) dw[i][j] = Frag<T>::mma(fb[j & 1], fa[i], dw[i][j], 0);
      }
    }
    if (next.e != now.e) {
      float* plane = p.part + int64_t(share + now.e) * p.plane;
#pragma unroll
      for (int i = 0; i < DM; ++i)
#pragma unroll
        for (int j = 0; j < DN; ++j) {
          const int m = am + 16 * i + (lane & 15), n = bn + 16 * j + 4 * (lane >> 4);
          if (m < p.out && n < p.in) *reinterpret_cast<f32x4*>(plane + int64_t(m) * p.in + n) = dw[i][j];
          dw[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
    now = next;
    next = later;
    ring = ring1;
  }
  rows_barrier<0>();
#endif
}

// Joins k_bwd_rows' planes: group e's are those of the shares its tiles are
// in, numbers share + e.
template <typename O>
__global__ __launch_bounds__(256) void k_join_rows(FusedArgs p, int bm, O* __restrict__ out, float* __restrict__ db) {
  const Span s = group_span(p.offsets, p.groups, p.rows, bm, blockIdx.y);
  const int64_t total = total_slots(p.offsets, p.groups, p.rows, bm);
  const int64_t size = int64_t(p.in) * p.out, all = size + p.out;
  const int shares = shares_in_use(total, p.shares);
  int lo = 0, n = 0;
  if (s.slots > 0) {
    lo = share_of(s.slot0, total, shares);
    n = share_of(s.slot0 + s.slots - 1, total, shares) - lo + 1;
  }
  __shared__ float box[256];
  for (int64_t i0 = int64_t(blockIdx.x) * 64; i0 < all; i0 += int64_t(gridDim.x) * 64) {
    const int64_t i = i0 + (threadIdx.x & 63);
    const float v = join_planes(p.part + int64_t(lo + int(blockIdx.y)) * p.plane + i, p.plane, n, i < all, box);
    if (threadIdx.x >= 64 || i >= all) continue;
    if (i < size)
      out[int64_t(blockIdx.y) * size + i] = O(v);
    else if (db != nullptr)
      db[int64_t(blockIdx.y) * p.out + (i - size)] = v;
  }
}

// --- launch ----------------------------------------------------------------------------------------

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Stretches of at most `unit` rows that `rows` rows in `groups` groups can make.
inline int64_t max_slots(int64_t rows, int32_t groups, int64_t unit) {
  if (groups == 0) return ceil_div(rows, unit);
  return rows / unit + std::min<int64_t>(groups, rows);
}

// Both operands in whole 16-byte chunks, near enough for 32-bit offsets.
template <typename T>
bool direct_ok(const ProductArgs& p, Mode mode) {
  const auto whole = [](const void* q, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % kChunk<T> == 0 && ld <= (1 << 20);
  };
  return whole(p.a, p.lda) && whole(p.b, p.ldb) && (mode == kDw || p.k % kChunk<T> == 0);
}

// Kernels of more than 64 KB of LDS have to ask for it, once per device.
template <class K>
void ask_lds(K kernel, int bytes, std::atomic<uint64_t>& asked) {
  int dev = 0;
  (void)hipGetDevice(&dev);
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if ((asked.load(std::memory_order_relaxed) & bit) == 0) {
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
}

template <typename T, Mode MODE, int BM, int BN, int WM, int WN, bool DIRECT, int KW>
void go_tile(const ProductArgs& p, int64_t grid, hipStream_t st) {
  constexpr int most = product_lds(BM, BN, WM, WN, KW, DIRECT);
  if constexpr (most > 65536) {
    static std::atomic<uint64_t> asked{0};
    ask_lds(&k_product<T, MODE, BM, BN, WM, WN, DIRECT, KW>, most, asked);
  }
  // a single step needs one stage, and leaves LDS for more workgroups (21,856 rows
  // 48 -> 768 fp16 with everything in the epilogue 35 -> 25 us)
  const bool staged = DIRECT && (MODE == kDw || KW > 1 || p.k > kStep<T>);
  k_product<T, MODE, BM, BN, WM, WN, DIRECT, KW>
      <<<int(grid), 64 * WM * WN * KW, product_lds(BM, BN, WM, WN, KW, staged), st>>>(p);
}

// Tiles of the product and the shape of its grid.
template <Mode MODE>
int64_t lay_out(ProductArgs& p, int bm, int bn) {
  p.tiles_n = int32_t(ceil_div(p.n, bn));
  if (MODE == kDw) {
    p.tiles = int32_t(ceil_div(p.m, bm)) * p.tiles_n;
    return (p.part != nullptr ? max_slots(p.rows, p.groups, p.unit) : std::max(1, p.groups)) * p.tiles;
  }
  p.unit = bm;
  p.tiles = p.tiles_n;
  return max_slots(p.rows, p.groups, bm) * p.tiles_n;
}

template <typename T, Mode MODE, int BM, int BN, int WM, int WN, int KW = 1>
void go_product(ProductArgs p, hipStream_t st) {
  const int64_t grid = lay_out<MODE>(p, BM, BN);
  if (direct_ok<T>(p, MODE))
    go_tile<T, MODE, BM, BN, WM, WN, true, KW>(p, grid, st);
  else if constexpr (BM <= 128 && BN <= 128)
    go_tile<T, MODE, BM, BN, WM, WN, false, KW>(p, grid, st);
}

// Wave sets that share the k steps of a tile: for few tiles and a k of
// eight steps at least.
template <typename T>
int wave_sets(int64_t tiles64, int64_t k) {
  if (k < 8 * kStep<T> || tiles64 > 512) return 1;
  return tiles64 <= 64 ? 8 : 4;
}

// k_rows: a short k, whole chunks everywhere, and rows enough that every
// workgroup walks several tiles for each time it fetches its weights.  Forward,
// bf16, gelu, this kernel against tiles, us:
//   rows      64 -> 64     64 -> 256    128 -> 128   256 -> 256
//   32,768    9.0   9.0    11.8  11.6   10.5  10.0   17.7  16.1
//   65,536    9.3   8.7    16.2  18.0   14.2  12.5   26.9  28.4
//   131,072   12.3  10.6   26.4  29.0   21.9  22.9   41.7  49.3
//   262,144   19.8  17.7   42.8  51.1   32.2  39.4   74.9  94.2
// and the same on 64 ragged groups:
//   65,536    14.1  9.5    26.7  22.4   18.6  20.4   37.4  37.3
//   262,144   22.9  22.1   48.8  59.8   37.7  49.5   83.3  117.6
// So the bound by the k steps is near the crossing from 256 columns on; the
// tiles keep up to 2 us at 128 -> 128 and at 64 -> 64, and up to 5 us with many
// groups near the bound.
template <typename T, Mode MODE>
bool rows_ok(const ProductArgs& p) {
  const auto whole = [](const void* q, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % kChunk<T> == 0 && ld <= (1 << 20);
  };
  return direct_ok<T>(p, MODE) && p.k <= 4 * kStep<T> && p.n % 8 == 0 && whole(p.out, p.ldo) &&
         (p.z == nullptr || whole(p.z, p.ldz)) && (p.residual == nullptr || whole(p.residual, p.ldr)) &&
         p.rows >= 32768 * ceil_div(p.k, kStep<T>);
}

template <typename T, Mode MODE, int KS, int WM, int WN>
void go_rows(ProductArgs p, hipStream_t st) {
  constexpr int BM = 128 / KS;
  p.tiles_n = int32_t(ceil_div(p.n, WN * 32));
  const int64_t most = max_slots(p.rows, p.groups, BM);
  const int shares = int(std::min<int64_t>(most, std::max(1, 512 / p.tiles_n)));   // two workgroups a CU
  k_rows<T, MODE, KS, WM, WN><<<shares * p.tiles_n, 512, 0, st>>>(p, shares);
}

// 256 x 256, a workgroup a CU: where the last round of them is mostly full and
// little of a tile lies past the columns (300,000 rows 512 -> 64 bf16: 107 us,
// 64 x 64 tiles 77 us).  fp32 has its matrix rate, a sixteenth, as the
// bound at any tile, and 64 x 64 leave the least of it to empty columns
// (20,000 rows 1024 -> 1024, 316 tiles of 256 x 256: 508 us, 337 us of 64 x 64).
// A tile's rows are of one group, so groups have to fill it on average.
// `filled`: other work fills the last round, which may be as empty as it likes
// (k_bwd_groups: 32,768 rows on 8 heads 512 -> 512 bf16, 272 tiles: the whole
// backward 158 us -> 136).
template <typename T, Mode MODE>
bool wide_rows(const ProductArgs& p, bool filled) {
  const int64_t across = ceil_div(p.n, 256), large = max_slots(p.rows, p.groups, 256) * across;
  const bool full = (filled || 4 * large >= 3 * ceil_div(large, 256) * 256) && 4 * p.n >= 3 * across * 256;
  return large >= 200 && full && p.rows / std::max(1, p.groups) >= 256 && p.k >= 512 && direct_ok<T>(p, MODE);
}

template <typename T, Mode MODE>
void run_rows(const ProductArgs& p, hipStream_t st) {
  if (rows_ok<T, MODE>(p)) {
    const int steps = int(ceil_div(p.k, kStep<T>));
    if (steps > 2) return p.n <= 128 ? go_rows<T, MODE, 4, 2, 4>(p, st) : go_rows<T, MODE, 4, 1, 8>(p, st);
    if (steps == 2)
      return p.n <= 64    ? go_rows<T, MODE, 2, 4, 2>(p, st)
             : p.n <= 128 ? go_rows<T, MODE, 2, 2, 4>(p, st)
                          : go_rows<T, MODE, 2, 1, 8>(p, st);
    return p.n <= 64    ? go_rows<T, MODE, 1, 4, 2>(p, st)
           : p.n <= 128 ? go_rows<T, MODE, 1, 2, 4>(p, st)
                        : go_rows<T, MODE, 1, 1, 8>(p, st);
  }
  if constexpr (sizeof(T) == 2) {
    if (wide_rows<T, MODE>(p, false)) {
      go_product<T, MODE, 256, 256, 2, 4>(p, st);
      return;
    }
    if (max_slots(p.rows, p.groups, 128) * ceil_div(p.n, 128) >= 256 && p.n > 64 && p.rows / std::max(1, p.groups) >= 96) {
      go_product<T, MODE, 128, 128, 2, 2>(p, st);
      return;
    }
  }
  const int sets = wave_sets<T>(max_slots(p.rows, p.groups, 64) * ceil_div(p.n, 64), p.k);
  if (sets == 8)
    go_product<T, MODE, 32, 32, 1, 1, 8>(p, st);
  else if (sets == 4)
    go_product<T, MODE, 64, 64, 2, 2, 4>(p, st);
  else
    go_product<T, MODE, 64, 64, 2, 2>(p, st);
}

// How the backward pass is cut: from the sizes alone, so that the workspace
// can be sized for it.
struct BwdPlan {
  bool fused;              // k_bwd_rows may run (the alignment decides), of so many steps and shares
  int32_t ko, ki, shares;
  bool small;              // dx and dw in one launch of 64 x 64 tiles
  bool sets;               // and that of 32 x 32 tiles of eight wave sets
  bool apart;              // dx by itself, in such tiles
  int32_t side_w;          // tile of dw
  int32_t unit_b, unit_w;  // rows of a stretch of db (with an activation) and of dw
  bool part_b, part_w;     // more than one stretch a group: partial sums to join
  int64_t plane;           // values of a plane of dw
  size_t dz, db, dw, total;
};
inline int64_t dz_ld(int32_t out, int chunk) { return ceil_div(out, chunk) * chunk; }

// dw in 256 x 256 tiles: 16-bit types, little of the edge tiles empty, and
// rows enough for a workgroup a CU.
template <typename T>
bool wide_dw(int64_t rows, int32_t in, int32_t out, int32_t groups) {
  const int64_t tiles = ceil_div(out, 256) * ceil_div(in, 256);
  return sizeof(T) == 2 && out % 8 == 0 && in % 8 == 0 && 4 * int64_t(out) * in >= 3 * tiles * 65536 &&
         rows * tiles >= 256 * 512;
}

template <typename T>
BwdPlan bwd_plan(int64_t rows, int32_t in, int32_t out, int32_t groups, int act) {
  BwdPlan s{};
  const int64_t slots = max_slots(rows, groups, 128);
  const auto steps = [](int32_t n) { return n <= 64 ? 1 : n <= 128 ? 2 : n <= 256 ? 4 : 8; };
  s.ko = steps(out);
  s.ki = steps(in);
  // One pass against slope, dx, dw and joins apart, bf16, gelu, us (without
  // groups; on 64; on 256):
  //   rows      64 -> 64     128 -> 128   256 -> 256
  //   16,384    18.5  21.1   24.6  25.6   41.3  38.6
  //   32,768    17.8  32.1   26.2  42.0   50.0  63.1
  //             31.1  29.6   45.0  41.1   90.7  58.8   on 64
  //             47.0  35.2   73.3  48.3   161   90     on 256
  //   131,072   29.5  59.0   46.7  88.9   112   159
  //             44.0  56.0   67.5  99.4   155   212    on 64
  //             62.2  73.5   98.4  125    253   179    on 256
  // Every group adds a plane of sums, written and read again, which the bound
  // does not count: with many groups for the rows the parts would be faster.
  s.fused = sizeof(T) == 2 && s.ko <= 4 && s.ki <= 4 && in % 8 == 0 && out % 8 == 0 && rows >= 32768;
  s.shares = 256;   // a workgroup a CU
  // (to 1024 tiles of 128 x 128 where both sides are narrow: 16384 rows 256 -> 256 bf16
  // with gelu 44 -> 37 us; 20,000 rows 777 -> 777 would take 254 us instead of 209)
  const int64_t few = std::max(in, out) <= 256 ? 1024 : 256;
  s.small = slots * ceil_div(in, 128) < few && slots * ceil_div(out, 128) < few;
  const int64_t x_tiles = max_slots(rows, groups, 64) * ceil_div(in, 64);
  const int64_t w_tiles = ceil_div(out, 64) * ceil_div(in, 64) * std::max(1, groups);
  // Small problems: steps one after the other at about 1 us each, in 64 x 64
  // tiles, three workgroups a CU (dw cut to 4 steps and joined by another
  // launch), or in 32 x 32 tiles of eight sets, one workgroup a CU; both
  // products alike in one launch, or dx in small tiles by itself (1 x 4096 ->
  // 4096: 48 us in one launch, 34 us in two)
  const int64_t heads = std::max(1, groups), x_steps = ceil_div(out, kStep<T>);
  const int64_t w_steps = ceil_div(ceil_div(rows, std::min<int64_t>(heads, std::max<int64_t>(1, rows))), kStep<T>);
  const int64_t launch = 6, join = w_steps > 4 ? launch : 0, w_cut = std::min<int64_t>(w_steps, 4);
  const int64_t x32 = (2 + ceil_div(x_steps, 8)) * ceil_div(4 * x_tiles, 256);
  const int64_t both64 = join + std::max(x_steps, w_cut) * ceil_div(x_tiles + w_tiles, 768);
  const int64_t both32 = (2 + ceil_div(std::max(x_steps, w_steps), 8)) * ceil_div(4 * (x_tiles + w_tiles), 256);
  const int64_t apart = launch + join + x32 + w_cut * ceil_div(w_tiles, 768);
  s.sets = s.small && both32 <= std::min(both64, apart);
  s.apart = s.small && !s.sets && apart < both64;
  // a side of at most 64 would leave half of a 128 tile empty (50,001 rows, 251 ->
  // 59 fp32: dw 61 us of 128 x 128, 40 us of 64 x 64)
  s.side_w = s.sets ? 32 : s.small || sizeof(T) == 4 || std::min(in, out) <= 64 ? 64 : 128;
  if (s.side_w == 128 && wide_dw<T>(rows, in, out, groups)) s.side_w = 256;
  const int64_t tiles = ceil_div(out, s.side_w) * ceil_div(in, s.side_w);
  // stretches so that about 768 workgroups (of 256 x 256: 256, one a CU) share the rows, of 4 k steps a set at least
  const int64_t cut = ceil_div(rows * tiles, s.side_w == 256 ? 256 : 768);
  int64_t unit = std::max<int64_t>((s.sets ? 32 : 4) * kStep<T>, ceil_div(cut, 64) * 64);
  // groups enough by themselves: only those of over twice the mean are cut
  if (groups * tiles >= (s.side_w == 256 ? 192 : 512))
    unit = std::max<int64_t>(unit, ceil_div(2 * rows, int64_t(groups) * 64) * 64);
  s.unit_w = int32_t(std::min<int64_t>(unit, 1 << 30));
  s.part_w = rows > s.unit_w;
  s.plane = ceil_div(int64_t(out) * in + out, 64) * 64;
  // about 2048 workgroups of the slope's kernel, 16 rows at least (4096 rows 256 ->
  // 256 bf16 with gelu, the whole backward: 38 us with 64, whose rows wait on each
  // other, 22 us with 16)
  const int64_t across = ceil_div(out, 64 * kChunk<T>);
  s.unit_b = int32_t(std::max<int64_t>(16, ceil_div(ceil_div(rows * across, 2048), 16) * 16));
  s.part_b = rows > s.unit_b;
  // (a fused pass writes no dz, but whether it runs is up to the alignment of
  // the call's operands)
  s.dz = act == kActNone ? 0 : align_up(size_t(rows) * dz_ld(out, kChunk<T>) * sizeof(T), 256);
  s.db = !s.part_b ? 0 : align_up(size_t(max_slots(rows, groups, s.unit_b)) * out * 4, 256);
  s.dw = !s.part_w ? 0 : align_up(size_t(max_slots(rows, groups, s.unit_w)) * s.plane * 4, 256);
  if (s.fused) s.dw = std::max(s.dw, size_t(s.shares + std::max(1, groups)) * s.plane * 4);
  s.total = s.dz + s.db + s.dw;
  return s;
}

template <typename T>
hipError_t linear_fwd(const LinearArgs& a, hipStream_t st) {
  ProductArgs p{};
  p.a = a.x;
  p.lda = a.ldx;
  p.b = a.w;
  p.ldb = a.ldw;
  p.b_group = int64_t(a.out) * a.ldw;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.groups = a.groups;
  p.n = a.out;
  p.k = a.in;
  p.bias = a.bias;
  p.residual = a.residual;
  p.ldr = a.ldr;
  p.out = a.y;
  p.ldo = a.ldy;
  p.z = a.z;
  p.ldz = a.ldz;
  p.act = a.act;
  run_rows<T, kFwd>(p, st);
  return hipGetLastError();
}

template <typename T>
hipError_t linear_bwd(const LinearArgs& a, char* ws, hipStream_t st) {
  const BwdPlan plan = bwd_plan<T>(a.rows, a.in, a.out, a.groups, a.act);
  if constexpr (sizeof(T) == 2) {
    const auto whole = [](const void* q, int64_t ld) {
      return q != nullptr && (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % 8 == 0 && ld <= (1 << 20);
    };
    if (plan.fused && a.dw != nullptr && (a.dx == nullptr || whole(a.dx, a.lddx)) && whole(a.dy, a.lddy) &&
        whole(a.x, a.ldx) && (a.act == kActNone || whole(a.z, a.ldz))) {
      FusedArgs f{};
      f.dy = a.dy;
      f.z = a.act == kActNone ? nullptr : a.z;
      f.x = a.x;
      f.w = a.w;
      f.dx = a.dx;
      f.part = reinterpret_cast<float*>(ws + plan.dz + plan.db);
      f.offsets = a.offsets;
      f.lddy = a.lddy;
      f.ldz = a.ldz;
      f.ldx = a.ldx;
      f.ldw = a.ldw;
      f.lddx = a.lddx;
      f.w_group = int64_t(a.out) * a.ldw;
      f.plane = plan.plane;
      f.rows = a.rows;
      f.groups = a.groups;
      f.in = a.in;
      f.out = a.out;
      f.act = a.act;
      f.shares = plan.shares;
      const auto go = [&](auto ko, auto ki) {
        k_bwd_rows<T, decltype(ko)::value, decltype(ki)::value><<<plan.shares, 512, 0, st>>>(f);
      };
      const auto go_in = [&](auto ko) {
        using std::integral_constant;
        if (plan.ki == 4)
          go(ko, integral_constant<int, 4>{});
        else if (plan.ki == 2)
          go(ko, integral_constant<int, 2>{});
        else
          go(ko, integral_constant<int, 1>{});
      };
      if (plan.ko == 4)
        go_in(std::integral_constant<int, 4>{});
      else if (plan.ko == 2)
        go_in(std::integral_constant<int, 2>{});
      else
        go_in(std::integral_constant<int, 1>{});
      const int bm = 128 / std::max(plan.ko, plan.ki);
      const dim3 grid(int(std::min<int64_t>(ceil_div(int64_t(a.out) * a.in + a.out, 64), std::max(16, 4096 / std::max(1, a.groups)))),
                      std::max(1, a.groups));
      if (a.dw_f32)
        k_join_rows<float><<<grid, 256, 0, st>>>(f, bm, static_cast<float*>(a.dw), a.db);
      else
        k_join_rows<T><<<grid, 256, 0, st>>>(f, bm, static_cast<T*>(a.dw), a.db);
      return hipGetLastError();
    }
  }
  T* dz = reinterpret_cast<T*>(ws);
  const bool slope = a.act != kActNone;
  const int groups = std::max(1, a.groups);
  // without rows only the zeros of dw and db are left to write
  const bool any = a.rows > 0;

  // db comes out of dw's product, but with an activation (or without dw) out
  // of the slope's pass
  const bool own_db = slope || a.dw == nullptr;
  DbJoin j{};
  if (any && (slope || (own_db && a.db != nullptr))) {
    int lanes = 1;
    while (lanes < 64 && lanes * kChunk<T> < a.out) lanes *= 2;
    const bool parts = a.db != nullptr && plan.part_b;
    float* part = reinterpret_cast<float*>(ws + plan.dz);
    // stretches as planned for the partial sums (unread where many rows come
    // without db); few rows: the groups themselves
    const bool cut = plan.part_b;
    k_act_grad<T><<<dim3(int(cut ? max_slots(a.rows, a.groups, plan.unit_b) : groups),
                         int(ceil_div(a.out, lanes * kChunk<T>))),
                    256, 0, st>>>(static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.z), a.ldz,
                                  slope ? dz : nullptr, dz_ld(a.out, kChunk<T>), a.offsets, a.groups, a.rows,
                                  plan.unit_b, a.out, a.act, lanes, cut ? part : nullptr, a.db);
    if (parts) {
      // one group has many partial rows, each of many groups few
      const int32_t cols = groups >= 16 ? 64 : 16;
      j = DbJoin{part, a.db, a.out, plan.unit_b, cols, int32_t(ceil_div(a.out, cols))};
    }
  }

  ProductArgs p{};
  p.a = slope ? dz : a.dy;
  p.lda = slope ? dz_ld(a.out, kChunk<T>) : a.lddy;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.groups = a.groups;
  ProductArgs x = p, w = p;
  x.b = a.w;
  x.ldb = a.ldw;
  x.b_group = int64_t(a.out) * a.ldw;
  x.n = a.in;
  x.k = a.out;
  x.out = a.dx;
  x.ldo = a.lddx;
  w.b = a.x;
  w.ldb = a.ldx;
  w.m = a.out;
  w.n = a.in;
  w.unit = plan.unit_w;
  w.out = a.dw;
  w.out_f32 = a.dw_f32;
  w.ldo = a.in;
  w.part = plan.part_w ? reinterpret_cast<float*>(ws + plan.dz + plan.db) : nullptr;
  w.plane = plan.plane;
  w.db = own_db && any ? nullptr : a.db;
  bool want_dx = a.dx != nullptr && any;
  const bool want_dw = a.dw != nullptr || (w.db != nullptr && !any);
  if (plan.small) {
    const int side = plan.side_w;
    if (plan.apart && want_dx) go_product<T, kDx, 32, 32, 1, 1, 8>(x, st);
    const bool here = want_dx && !plan.apart;
    const int64_t x_tiles = here ? lay_out<kDx>(x, side, side) : 0;
    const int64_t w_tiles = want_dw ? lay_out<kDw>(w, side, side) : 0;
    const int64_t grid = x_tiles + w_tiles + int64_t(j.blocks) * groups;
    if (grid > 0) {
      const bool direct = (!here || direct_ok<T>(x, kDx)) && (!want_dw || direct_ok<T>(w, kDw));
      const auto go = [&](auto d, auto sets) {
        constexpr bool D = decltype(d)::value, S = decltype(sets)::value;
        constexpr int TILE = S ? 32 : 64, W = S ? 1 : 2, KW = S ? 8 : 1, lds = product_lds(TILE, TILE, W, W, KW, D);
        if constexpr (lds > 65536) {
          static std::atomic<uint64_t> asked{0};
          ask_lds(&k_bwd<T, TILE, W, D, KW>, lds, asked);
        }
        k_bwd<T, TILE, W, D, KW><<<int(grid), 64 * W * W * KW, lds, st>>>(x, int(x_tiles), w, int(w_tiles), j);
      };
      if (direct)
        plan.sets ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
      else
        plan.sets ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    }
  } else {
    if (j.blocks > 0) k_join_db<<<j.blocks * groups, 256, 0, st>>>(j, p);
    bool want_w = want_dw;
    if constexpr (sizeof(T) == 2) {
      if (want_dx && want_dw && a.groups > 0 && plan.side_w == 256 && wide_rows<T, kDx>(x, true) && direct_ok<T>(w, kDw)) {
        const int64_t w_grid = lay_out<kDw>(w, 256, 256), x_grid = lay_out<kDx>(x, 256, 256);
        constexpr int lds = product_lds(256, 256, 2, 4, 1, true);
        static std::atomic<uint64_t> asked{0};
        ask_lds(&k_bwd_groups<T>, lds, asked);
        k_bwd_groups<T><<<int(w_grid + x_grid), 512, lds, st>>>(x, w, int(w_grid));
        want_dx = want_w = false;
      }
    }
    if (want_dx) run_rows<T, kDx>(x, st);
    if (want_w && plan.side_w == 64)
      go_product<T, kDw, 64, 64, 2, 2>(w, st);
    if constexpr (sizeof(T) == 2) {
      if (want_w && plan.side_w == 256 && direct_ok<T>(w, kDw))
        go_product<T, kDw, 256, 256, 2, 4>(w, st);
      else if (want_w && plan.side_w != 64)
        go_product<T, kDw, 128, 128, 2, 2>(w, st);
    }
  }
  if (want_dw && w.part != nullptr) {
    const int64_t size = int64_t(a.out) * a.in;
    const dim3 grid(int(std::min<int64_t>(ceil_div(size + a.out, 64), std::max(16, 4096 / groups))), groups);
    if (a.dw_f32)
      k_join<float><<<grid, 256, 0, st>>>(w.part, w.plane, a.offsets, a.groups, a.rows, plan.unit_w, size,
                                          static_cast<float*>(a.dw), a.out, w.db);
    else
      k_join<T><<<grid, 256, 0, st>>>(w.part, w.plane, a.offsets, a.groups, a.rows, plan.unit_w, size,
                                      static_cast<T*>(a.dw), a.out, w.db);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace net
}  // namespace gs
