// The gate: the k largest logits of a row with their softmax weights, and the
// gradient of the logits.
//
//   forward   k times the largest logit left, ties to the lower index; weights
//             e^(l - m) / sum e^(l - m), m the largest, the sum over the chosen
//             (renorm) or over all
//   backward  renorm: dl = w (dw - s) where chosen, s = sum w dw; else
//             dl = [chosen] w dw - p s, p = w_0 e^(l - l_0), 0 the first choice:
//             the row's maximum and sum are not worked out again (but for a row
//             without its first choice)
//
// A row lies in the registers of L lanes, read once.  A logit becomes an
// unsigned number that orders as it does, with its column below it, so that a
// maximum of numbers is the choice: 32 bits for 16-bit logits, 64 for fp32.
// The gradient's few chosen entries go through LDS to the lanes that hold
// their columns.  Bound by the bytes of the logits, with the vector unit about
// as busy: the instructions of the loops over the logits count.  1,000,000 x 64
// bf16, 2 choices: 29 us (144 MB at 5.0 TB/s); gradient of 70,001 x 250 fp32, 8
// choices, of all logits: 32 us (147 MB at 4.5 TB/s).  With 8 choices the vector
// unit bounds it: bf16 x 64 39 us, x 256 130, fp32 x 64 72, x 256 264.  The gradient
// over the chosen reads no logits and is bound by LDS: 1,000,000 x 64 bf16, 2
// choices, 51 us, of which LDS is busy 42, most of it conflicts of banks (152 MB
// take 30); over all logits 68 us.
#include <algorithm>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;

// A logit's bits as a number: its magnitude, negated under a sign, plus that of
// infinity, without sign.  Minus infinity becomes 0, zeros of either sign the
// same; NaN of either sign comes out above infinity (a negative one by wrapping
// around).  16-bit logits two at a time.
typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// What is compared: the number, then the lower column.  Below kOne: minus
// infinity, or (0) no logit.
template <typename T>
struct Pick {      // fp32
  using U = uint64_t;
  static constexpr U kOne = U(1) << 32;
  static constexpr int32_t kInf = 0x7F800000;
  static __device__ __forceinline__ void make(const Chunk<float>& v, int col, U (&u)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t b = __builtin_bit_cast(int32_t, v.v[i]);
      const uint32_t m = uint32_t(b >> 31);
      u[i] = U(((uint32_t(b) & 0x7FFFFFFFu) ^ m) - m + uint32_t(kInf)) << 32 | uint32_t(0xFFFF - col - i);
    }
  }
  static __device__ __forceinline__ float value(U u) {
    const uint32_t s = uint32_t(u >> 32) - uint32_t(kInf), m = uint32_t(int32_t(s) >> 31);
    return __builtin_bit_cast(float, ((s ^ m) - m) | (s & 0x80000000u));
  }
};
template <typename T, uint16_t kInf>
struct Pick16 {
  using U = uint32_t;
  static constexpr U kOne = 0x10000u;
  static __device__ __forceinline__ void make(const Chunk<T>& v, int col, U (&u)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      u16x2 b;
      __builtin_memcpy(&b, &v.v[i], 4);
      const u16x2 m = __builtin_bit_cast(u16x2, __builtin_bit_cast(s16x2, b) >> s16x2{15, 15});
      const u16x2 n = ((b & u16x2{0x7FFF, 0x7FFF}) ^ m) - m + u16x2{kInf, kInf};
      uint32_t both;
      __builtin_memcpy(&both, &n, 4);
      u[i] = both << 16 | uint32_t(0xFFFF - col - i);
      u[i + 1] = (both & 0xFFFF0000u) | uint32_t(0xFFFF - col - i - 1);
    }
  }
  // the logit's bits as the upper half of a word
  static __device__ __forceinline__ uint32_t bits(U u) {
    const uint32_t s = (u & 0xFFFF0000u) - (uint32_t(kInf) << 16), m = uint32_t(int32_t(s) >> 31);
    return ((s ^ m) - m) | (s & 0x80000000u);
  }
};
template <>
struct Pick<bf16> : Pick16<bf16, 0x7F80> {
  static __device__ __forceinline__ float value(U u) { return __builtin_bit_cast(float, bits(u)); }
};
template <>
struct Pick<f16> : Pick16<f16, 0x7C00> {
  static __device__ __forceinline__ float value(U u) {
    return float(__builtin_bit_cast(f16, uint16_t(bits(u) >> 16)));
  }
};
__device__ __forceinline__ int column_of(uint64_t u) { return 0xFFFF - int(uint32_t(u) & 0xFFFFu); }

template <typename U>
__device__ __forceinline__ U larger(U a, U b) {
  return a > b ? a : b;
}

// op(v, w) with w that of a lane whose number differs in one bit (d: 1, 2, 16,
// 32) or, for 4 and 8, of one in the other 4 or 8 lanes, which is as good for a
// maximum or sum of lanes that agree so far.  All in the vector unit: within 16
// lanes by their rows' patterns, beyond by exchanging rows of two copies.
template <int d, typename Op>
__device__ __forceinline__ uint32_t with_other(uint32_t v, Op op) {
  if constexpr (d == 1) return op(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true)));
  if constexpr (d == 2) return op(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true)));
  if constexpr (d == 4) return op(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x141, 0xF, 0xF, true)));   // mirror of 8
  if constexpr (d == 8) return op(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x140, 0xF, 0xF, true)));   // of 16
  if constexpr (d == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return op(uint32_t(r[0]), uint32_t(r[1]));
  }
  if constexpr (d == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op(uint32_t(r[0]), uint32_t(r[1]));
  }
}
template <int L, int d = 1, typename Op>
__device__ __forceinline__ uint32_t row_all(uint32_t v, Op op) {
  if constexpr (d < L)
    return row_all<L, 2 * d>(with_other<d>(v, op), op);
  else
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return row_all<L>(v, larger<uint32_t>);
}
// The upper halves' maximum, then that of the lower halves that go with it; of
// a whole wave usually one lane's.
template <int L>
__device__ __forceinline__ uint64_t row_max(uint64_t v) {
  const uint32_t upper = row_max<L>(uint32_t(v >> 32));
  if constexpr (L == 64) {
    const uint64_t has = __builtin_amdgcn_ballot_w64(uint32_t(v >> 32) == upper);
    if ((has & (has - 1)) == 0)
      return uint64_t(upper) << 32 | uint32_t(__builtin_amdgcn_readlane(int(v), __builtin_ctzll(has)));
  }
  return uint64_t(upper) << 32 | row_max<L>(uint32_t(v >> 32) == upper ? uint32_t(v) : 0u);
}
template <int L>
__device__ __forceinline__ float row_max_of(float v) {
  return __builtin_bit_cast(float, row_all<L>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
                              return __builtin_bit_cast(
                                  uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
                            }));
}
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  return __builtin_bit_cast(float, row_all<L>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
                              return __builtin_bit_cast(
                                  uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                            }));
}

// 4 or 8 numbers in descending order: pairs, halves, and their merge (Batcher's
// odd-even network).
template <int N, typename U>
__device__ __forceinline__ void sort_down(U (&v)[N]) {
  auto order = [&](int i, int j) {
    const U a = larger(v[i], v[j]);
    v[j] = v[i] < v[j] ? v[i] : v[j];
    v[i] = a;
  };
#pragma unroll
  for (int h = 0; h < N; h += 4) {
    order(h, h + 1), order(h + 2, h + 3);
    order(h, h + 2), order(h + 1, h + 3);
    order(h + 1, h + 2);
  }
  if constexpr (N == 8) {
    order(0, 4), order(1, 5), order(2, 6), order(3, 7);
    order(2, 4), order(3, 5);
    order(1, 2), order(3, 4), order(5, 6);
  }
}

// e^x, x <= 0 or NaN: the native exp2 of the rounded product with log2 e, and
// what that rounding left out (2^-22 of the result in all).
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * 1.44269504088896340736f;
  const float rest = fmaf(x, 1.92596299112661746887e-8f, fmaf(x, 1.44269504088896340736f, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return y < -200.0f ? 0.0f : fmaf(e, rest * 0.69314718055994530942f, e);
}

// Which chunks a lane holds.  kExact: every lane's lie inside the row.  Else
// one past the row's end is moved back onto it, and what another chunk has is
// masked; kNarrow: a row of less than a chunk.
enum Fit { kExact, kMoved, kNarrow };

// Lane l's chunks of a row, all asked for before the first is waited for.
template <typename T, int L, int C, Fit F>
struct Held {
  Chunk<T> v[C];
  __device__ __forceinline__ static int first(int l, int j) { return (l + L * j) * kChunk<T>; }
  __device__ __forceinline__ static int at(int l, int j, int groups) {
    return F == kNarrow ? 0 : F == kExact ? first(l, j) : std::min(first(l, j), groups - kChunk<T>);
  }
  // whether no other chunk has the i-th of chunk j, and the row does
  __device__ __forceinline__ static bool own(int l, int j, int i, int groups) {
    return F == kNarrow ? i < groups : i >= first(l, j) - at(l, j, groups);
  }
  __device__ __forceinline__ void load(const GateArgs& a, int64_t r, int l) {
    const T* __restrict__ x = static_cast<const T*>(a.logits) + r * a.ld;
#pragma unroll
    for (int j = 0; j < C; ++j)
      v[j] = F == kNarrow ? load_chunk_n(x, a.groups) : load_whole(x + at(l, j, a.groups));
  }
};

// Choices (rounded up) for which a lane sorts its numbers: from 4 where that
// saves looking through several chunks, or 64-bit numbers (1,000,000 x 256 bf16,
// k 4, four chunks a lane 109 us sorted; one chunk unsorted 167).
template <typename T>
constexpr bool many_choices(int chunks, int km) {
  return km >= (sizeof(T) == 4 || chunks > 1 ? 4 : 8);
}

// L lanes a row, C chunks a lane; KM: choices, rounded up.
template <typename T, int L, int C, int KM, Fit F>
__device__ __forceinline__ void gate_row(const GateArgs& a, int64_t r, int l, const Held<T, L, C, F>& x) {
  constexpr int K = kChunk<T>;
  using P = Pick<T>;
  using U = typename P::U;
  U mine[C][K];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int at = x.at(l, j, a.groups);
    U u[K];
    P::make(x.v[j], at, u);
#pragma unroll
    for (int i = 0; i < K; ++i)
      mine[j][i] = F != kExact && !x.own(l, j, i, a.groups) ? U(0) : u[i];
  }
  // With its chunks in descending order a lane's next choice is one of their
  // first numbers, and a choice moves that chunk's others up; otherwise a choice
  // is looked for and taken out among all of them, which is less for few choices.
  constexpr bool kSorted = many_choices<T>(C, KM);
  if constexpr (kSorted)
#pragma unroll
    for (int j = 0; j < C; ++j) sort_down<K>(mine[j]);
  // choice q is lane q's, modulo L, to weigh and to write
  constexpr int Q = (KM + L - 1) / L;
  U pick[Q] = {};
  float top = 0.0f, total = 0.0f;
#pragma unroll
  for (int q = 0; q < KM; ++q) {
    U best = mine[0][0];
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < (kSorted ? 1 : K); ++i) best = larger(best, mine[j][i]);
    best = row_max<L>(best);
    if (q == 0) {
      top = P::value(best);
      if (a.renorm == 0)
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const float e = exp_of(float(x.v[j].v[i]) - top);
            total += F != kExact && !x.own(l, j, i, a.groups) ? 0.0f : e;
          }
    }
    pick[q / L] = q < a.k && l == q % L ? best : pick[q / L];
    // columns are distinct, so one number is the choice
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const bool chosen = mine[j][0] == best;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (q + 1 == KM) continue;
        if constexpr (kSorted)
          mine[j][i] = chosen ? (i + 1 < K ? mine[j][i + 1 < K ? i + 1 : i] : U(0)) : mine[j][i];
        else
          mine[j][i] = mine[j][i] == best ? U(0) : mine[j][i];
      }
    }
  }
  float e[Q];
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    e[j] = pick[j] < P::kOne ? 0.0f : exp_of(P::value(pick[j]) - top);
    if (a.renorm != 0) total += e[j];
  }
  total = row_sum<L>(total);
  // 1 / total, total of at least 1: the reciprocal and one step of Newton's
  float share = __builtin_amdgcn_rcpf(total);
  share = fmaf(fmaf(-total, share, 1.0f), share, share);
#pragma unroll
  for (int j = 0; j < Q; ++j)
    if (j * L + l < a.k) {
      const bool none = pick[j] < P::kOne;
      a.ids[r * a.k + j * L + l] = none ? -1 : column_of(pick[j]);
      a.weights[r * a.k + j * L + l] = none ? 0.0f : e[j] * share;
    }
}

template <typename T, int L, int C, int KM, Fit F>
__device__ __forceinline__ void gate_row_bwd(const GateArgs& a, int64_t r, int l, const Held<T, L, C, F>& x,
                                             float* __restrict__ box) {
  constexpr int K = kChunk<T>, Q = (KM + L - 1) / L;      // choices of a lane
  T* __restrict__ dl = static_cast<T*>(a.dlogits) + r * a.lddl;
  int32_t id[Q];
  float part[Q], w[Q], s = 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int c = l + q * L;
    id[q] = c < a.k ? a.ids[r * a.k + c] : -1;
    if (uint32_t(id[q]) >= uint32_t(a.groups)) id[q] = -1;
    w[q] = id[q] < 0 ? 0.0f : a.weights[r * a.k + c];
    part[q] = id[q] < 0 ? 0.0f : w[q] * a.dweights[r * a.k + c];
    s += part[q];
  }
  // the row's part of the box, 0 but for the choices
  float* const mine = box + (threadIdx.x / L) * (L * C * K);
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < K; i += 4)
      *reinterpret_cast<f32x4*>(mine + x.first(l, j) + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  wave_sync();
  s = row_sum<L>(s);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (id[q] >= 0) atomicAdd(mine + id[q], a.renorm != 0 ? part[q] - w[q] * s : part[q]);
  const int base = threadIdx.x & 63 & ~(L - 1);
  float first = 0.0f, scale = 0.0f;
  if (a.renorm == 0) {
    const int32_t id0 = __shfl(id[0], base, 64);
    if (id0 >= 0) {
      first = float(static_cast<const T*>(a.logits)[r * a.ld + id0]);
      scale = -__shfl(w[0], base, 64) * s;
    } else {
      // no first choice: nothing was left to choose, or it was dropped since
      float most = -__builtin_inff(), total = 0.0f;
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (F == kExact || x.own(l, j, i, a.groups)) most = fmaxf(most, float(x.v[j].v[i]));
      most = row_max_of<L>(most);
      if (most > -__builtin_inff()) {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < K; ++i)
            if (F == kExact || x.own(l, j, i, a.groups)) total += exp_of(float(x.v[j].v[i]) - most);
        first = most;
        scale = -s / row_sum<L>(total);
      }
    }
  }
  wave_sync();
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int at = x.at(l, j, a.groups);
    Chunk<T> o;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float g = mine[at + i];
      if (a.renorm == 0) g = fmaf(scale, exp_of(float(x.v[j].v[i]) - first), g);
      o.v[i] = T(g);
    }
    // a chunk that was moved back writes what others write too
    if constexpr (F == kNarrow) {
      store_chunk_n(dl, o, a.groups);
    } else if (x.first(l, j) < a.groups) {
      store_chunk(dl + at, o);
    }
  }
  wave_sync();      // the next row's zeros
}

// Rows are walked with the next one's logits on their way: a row's work is
// longer than its loads, but a wave that starts with a load only waits.
template <typename T, int L, int C, int KM, Fit F, bool kFwd>
__global__ __launch_bounds__(kThreads) void k_gate(GateArgs a) {
  constexpr int kRows = kThreads / L;
  __shared__ __align__(16) float box[kFwd ? 4 : kThreads * C * kChunk<T>];
  const int l = threadIdx.x % L;
  const bool reads = kFwd || a.renorm == 0;
  Held<T, L, C, F> next;
  int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / L;
  if (r >= a.rows) return;
  if (reads) next.load(a, r, l);
  // all lanes of a row together
  for (; r < a.rows; r += int64_t(gridDim.x) * kRows) {
    const Held<T, L, C, F> x = next;
    if (reads) next.load(a, std::min<int64_t>(r + int64_t(gridDim.x) * kRows, a.rows - 1), l);
    if constexpr (kFwd)
      gate_row<T, L, C, KM, F>(a, r, l, x);
    else
      gate_row_bwd<T, L, C, KM, F>(a, r, l, x, box);
  }
}

template <typename T, int L, int C, int KM, Fit F, bool kFwd>
hipError_t go(const GateArgs& a, hipStream_t st) {
  // as many workgroups as are there at a time
  const int64_t blocks = std::min<int64_t>((int64_t(a.rows) + kThreads / L - 1) / (kThreads / L), 2048);
  k_gate<T, L, C, KM, F, kFwd><<<unsigned(blocks), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

// Choices in powers of two, up to those that such a row can have: no more than
// its columns, and with four chunks four a lane, as below.
template <typename T, int L, int C, Fit F, bool kFwd, int KM = 1>
hipError_t by_choices(const GateArgs& a, hipStream_t st) {
  constexpr int kColumns = F == kNarrow ? kChunk<T> - 1 : L * C * kChunk<T>;
  constexpr int kMost = std::min({int(kMaxChoices), kColumns, C == 4 ? 4 * L : int(kMaxChoices)});
  if constexpr (KM >= kMost)
    return go<T, L, C, KM, F, kFwd>(a, st);
  else
    return a.k <= KM ? go<T, L, C, KM, F, kFwd>(a, st) : by_choices<T, L, C, F, kFwd, 2 * KM>(a, st);
}

template <typename T, int L, int C, bool kFwd>
hipError_t by_fit(const GateArgs& a, hipStream_t st) {
  if constexpr (L * C > 1)      // a row of one chunk, and not less, is exact
    if (a.groups != L * C * kChunk<T>) return by_choices<T, L, C, kMoved, kFwd>(a, st);
  return by_choices<T, L, C, kExact, kFwd>(a, st);
}

// The forward pass: with four chunks a lane instead of one, four times as many
// rows share the exchanges between lanes (k 8, bf16 1,000,000 x 64 45 -> 39 us, x 256 206
// -> 129, fp32 x 64 103 -> 70, x 256 490 -> 262; k 2, bf16 x 64 30 -> 25, x 256 126 ->
// 101).  Not so where that leaves a SIMD less than four waves (20,000 x 256 bf16, k 16,
// 9 us with one chunk, 11 with four), a lane more than four choices to weigh
// (1,000,000 x 64 bf16, k 16, 71 us with 8 lanes, 85 with 2), or one lane alone (x 16
// fp32, k 8, 29 and 46).
template <typename T, int L, int C, bool kFwd>
hipError_t by_lanes(const GateArgs& a, int chunks, hipStream_t st) {
  if constexpr (kFwd && L * C >= 8)
    if (int64_t(a.rows) * chunks >= 4 * 64 * 4096 && a.k <= L * C) return by_fit<T, L * C / 4, 4, true>(a, st);
  return by_fit<T, L, C, kFwd>(a, st);
}

template <typename T, bool kFwd>
hipError_t by_width(const GateArgs& a, hipStream_t st) {
  const int chunks = (a.groups + kChunk<T> - 1) / kChunk<T>;
  // as many lanes as chunks: with 8 lanes for 16 bf16 logits six would be idle
  if (a.groups < kChunk<T>) return by_choices<T, 1, 1, kNarrow, kFwd>(a, st);
  if (chunks <= 1) return by_lanes<T, 1, 1, kFwd>(a, chunks, st);
  if (chunks <= 2) return by_lanes<T, 2, 1, kFwd>(a, chunks, st);
  if (chunks <= 4) return by_lanes<T, 4, 1, kFwd>(a, chunks, st);
  if (chunks <= 8) return by_lanes<T, 8, 1, kFwd>(a, chunks, st);
  if (chunks <= 16) return by_lanes<T, 16, 1, kFwd>(a, chunks, st);
  if (chunks <= 32) return by_lanes<T, 32, 1, kFwd>(a, chunks, st);
  if (chunks <= 64) return by_lanes<T, 64, 1, kFwd>(a, chunks, st);
  if constexpr (sizeof(T) == 4)
    if (chunks > 128) return by_fit<T, 64, 4, kFwd>(a, st);
  return by_lanes<T, 64, 2, kFwd>(a, chunks, st);
}

template <typename T>
hipError_t either(bool fwd, const GateArgs& a, hipStream_t st) {
  return fwd ? by_width<T, true>(a, st) : by_width<T, false>(a, st);
}

hipError_t by_type(int type, bool fwd, const GateArgs& a, hipStream_t st) {
  if (type == kTypeBF16) return either<bf16>(fwd, a, st);
  if (type == kTypeF16) return either<f16>(fwd, a, st);
  return either<float>(fwd, a, st);
}

}  // namespace
}  // namespace net

hipError_t launch_gate_fwd(int type, const GateArgs& a, hipStream_t st) { return net::by_type(type, true, a, st); }
hipError_t launch_gate_bwd(int type, const GateArgs& a, hipStream_t st) { return net::by_type(type, false, a, st); }

}  // namespace gs
