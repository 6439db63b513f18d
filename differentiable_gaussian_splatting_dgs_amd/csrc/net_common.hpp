// Shared by the network operators (layer_norm.hip, linear_*.hip): storage
// types, 16-byte chunks of a row at any alignment, the activations, and the
// search of a ragged group list.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gs_internal.h"

namespace gs {
namespace net {

using bf16 = __bf16;
using f16 = _Float16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Elements in a 16-byte chunk.
template <typename T>
constexpr int kChunk = int(16 / sizeof(T));

template <typename T>
struct alignas(16) Chunk {
  T v[kChunk<T>];
};

// gfx950 reads and writes 16 bytes at any element alignment in one
// instruction, so rows of odd length take the same path as aligned ones.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* __restrict__ p) {
  Chunk<T> c;
  __builtin_memcpy(&c, p, 16);
  return c;
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* __restrict__ p, const Chunk<T>& c) {
  __builtin_memcpy(p, &c, 16);
}
// The first n elements (the others 0; nothing past p + n is read).
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk_n(const T* __restrict__ p, int n) {
  if (n >= kChunk<T>) return load_chunk(p);
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < kChunk<T>; ++i) c.v[i] = i < n ? p[i] : T(0.0f);
  return c;
}
template <typename T>
__device__ __forceinline__ void store_chunk_n(T* __restrict__ p, const Chunk<T>& c, int n) {
  if (n >= kChunk<T>) {
    store_chunk(p, c);
    return;
  }
#pragma unroll
  for (int i = 0; i < kChunk<T>; ++i)
    if (i < n) p[i] = c.v[i];
}

// --- activations ----------------------------------------------------------------

// e^x and 1/x for 16-bit storage: the native exp2 and reciprocal.  The
// rounded argument of exp2 makes e^x off by about |x| 2^-23 of itself, beside
// the instruction's own 2^-22 (below 2^-16 up to |x| = 88, where fp32 ends;
// the half step is 2^-8 of bf16, 2^-11 of fp16); 1/x by 2^-22.  fp32 storage
// takes the library function and the IEEE division.
template <typename T>
__device__ __forceinline__ float exp_t(float x) {
  if constexpr (sizeof(T) == 4)
    return expf(x);
  else
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}
template <typename T>
__device__ __forceinline__ float rcp_t(float x) {
  if constexpr (sizeof(T) == 4)
    return 1.0f / x;
  else
    return __builtin_amdgcn_rcpf(x);
}

// Phi(v) = (1 + erf(v / sqrt 2)) / 2.  fp32 storage: erfcf, which keeps the
// relative error of the tail.  16-bit storage: Phi(-x) = 2^p(x) for x >= 0,
// p of degree 8 the minimax fit of log2 Phi(-x) on [0, 6.5] with the error
// weighted by max(Phi(-x), 10^-3) and p(0) = -1: 1.8e-7 off at most, 1.8e-4
// of itself in the tail; beyond 6.5 p keeps falling.  One exponential and
// no reciprocal: an epilogue that is bound by memory has room for about 20
// instructions a value (the mid decoder layer, 1,000,000 x 64 -> 256 with
// z: 345 us with an erf of one exponential, one reciprocal and five
// multiply-adds more, 324 us with this).
template <typename T>
__device__ __forceinline__ float normal_cdf(float v) {
  if constexpr (sizeof(T) == 4) {
    return 0.5f * erfcf(v * -0.70710678118654752440f);
  } else {
    const float x = fabsf(v);
    float p = fmaf(-4.37513261e-07f, x, 8.06129225e-06f);
    p = fmaf(p, x, -2.64287306e-05f);
    p = fmaf(p, x, -5.39061132e-04f);
    p = fmaf(p, x, 7.58801196e-03f);
    p = fmaf(p, x, -5.28385972e-02f);
    p = fmaf(p, x, -4.59110487e-01f);
    p = fmaf(p, x, -1.15111367e+00f);
    p = fmaf(p, x, -1.0f);
    const float tail = __builtin_amdgcn_exp2f(p);
    return v < 0.0f ? tail : 1.0f - tail;
  }
}

// NaN passes through every activation (relu compares instead of taking a
// maximum, which would drop it).
template <typename T>
__device__ __forceinline__ float act_apply(float v, int act) {
  if (act == kActRelu) return v < 0.0f ? 0.0f : v;
  if (act == kActSilu) return v * rcp_t<T>(1.0f + exp_t<T>(-v));
  if (act == kActGelu) return v * normal_cdf<T>(v);
  return v;
}
// gelu'(v) = Phi(v) + v phi(v).  16-bit storage: with x = |v|, gelu'(-x) =
// e^(-x^2 / 2) P(x) and gelu'(x) = 1 - gelu'(-x), P of degree 10 the minimax
// fit on [0, 6] with the error weighted by the exponential (5e-7 off at most):
// 20 instruction slots a value where Phi and phi take 23, in a pass that the
// slope of a 256-wide layer bounds.
template <typename T>
__device__ __forceinline__ float gelu_slope(float v) {
  if constexpr (sizeof(T) == 4) {
    const float density = 0.39894228040143267794f * expf(-0.5f * v * v);
    return fmaf(fminf(fmaxf(v, -64.0f), 64.0f), density, normal_cdf<T>(v));   // no infinity times 0
  } else {
    const float x = fminf(fabsf(v), 7.0f);
    const float e = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170368f);
    float p = fmaf(5.42516376e-07f, x, -1.54095325e-05f);
    p = fmaf(p, x, 1.90652152e-04f);
    p = fmaf(p, x, -1.37058932e-03f);
    p = fmaf(p, x, 6.5064465e-03f);
    p = fmaf(p, x, -2.22826763e-02f);
    p = fmaf(p, x, 5.94712761e-02f);
    p = fmaf(p, x, -1.31751587e-01f);
    p = fmaf(p, x, 2.49754565e-01f);
    p = fmaf(p, x, -7.97867768e-01f);
    p = fmaf(p, x, 0.5f);
    const float h = e * p;
    return v < 0.0f ? h : 1.0f - h;
  }
}

// act'(v); relu's is 0 at 0 and at NaN.
template <typename T>
__device__ __forceinline__ float act_slope(float v, int act) {
  if (act == kActRelu) return v > 0.0f ? 1.0f : 0.0f;
  if (act == kActSilu) {
    const float p = rcp_t<T>(1.0f + exp_t<T>(-v));
    return p * fmaf(v, 1.0f - p, 1.0f);
  }
  if (act == kActGelu) return gelu_slope<T>(v);
  return 1.0f;
}

// --- ragged groups -----------------------------------------------------------------

// One stretch of at most `unit` rows of one group.  Slots count stretches
// over all groups in order.
struct Span {
  int32_t e, row0, row1;      // group, rows
  int32_t slot0, slots;       // the group's first slot and how many it has
  int32_t end;                // the group's last row + 1
};

__device__ __forceinline__ int32_t clamp_row(int64_t v, int32_t rows) {
  return v < 0 ? 0 : (v > rows ? rows : int32_t(v));
}

// Bounds of the 64 groups from e0 on, one per lane: offsets clamped to
// [0, rows] and made non-decreasing by a running maximum (`carry`: the
// groups before), so that whatever the list holds, groups never overlap and
// never leave the rows.  `first`, `n`: the group's first slot and its slots
// (0 past the last group); `base`: slots of the groups before.  All lanes of
// a wave call it together.
__device__ __forceinline__ void group_block(const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                            uint32_t unit, int32_t e0, int32_t& carry, int32_t& base, int32_t& lo,
                                            int32_t& hi, int32_t& first, int32_t& n) {
  const int lane = threadIdx.x & 63;
  const int32_t e = e0 + lane;
  hi = e < groups ? clamp_row(offsets[e + 1], rows) : 0;
  hi = hi > carry ? hi : carry;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(hi, d, 64);
    if (lane >= d) hi = o > hi ? o : hi;
  }
  const int32_t below = __shfl_up(hi, 1, 64);
  lo = lane == 0 ? carry : below;
  n = int32_t((uint32_t(hi - lo) + unit - 1) / unit);
  int32_t sum = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  first = base + sum - n;
  base += __builtin_amdgcn_readlane(sum, 63);
  carry = __builtin_amdgcn_readlane(hi, 63);
}

// The span of slot t; e < 0: there is no such slot.  groups == 0: one group
// of all rows, no list.
__device__ __forceinline__ Span find_span(const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                          uint32_t unit, int32_t t) {
  if (groups == 0) {
    const int64_t r0 = int64_t(t) * unit;
    const int64_t r1 = r0 + unit < rows ? r0 + unit : rows;
    return Span{r0 < rows ? 0 : -1, int32_t(r0), int32_t(r1), 0, int32_t((uint32_t(rows) + unit - 1) / unit), rows};
  }
  int32_t carry = clamp_row(offsets[0], rows), base = 0;
  for (int32_t e0 = 0; e0 < groups; e0 += 64) {
    int32_t lo, hi, first, n;
    group_block(offsets, groups, rows, unit, e0, carry, base, lo, hi, first, n);
    const uint64_t m = __builtin_amdgcn_ballot_w64(t >= first && t < first + n);
    if (m == 0) continue;
    const int l = __builtin_ctzll(m);
    const int32_t s0 = __builtin_amdgcn_readlane(first, l), h0 = __builtin_amdgcn_readlane(hi, l);
    const int32_t r0 = __builtin_amdgcn_readlane(lo, l) + int32_t(uint32_t(t - s0) * unit);
    return Span{e0 + l, r0, uint32_t(h0 - r0) < unit ? h0 : r0 + int32_t(unit), s0, __builtin_amdgcn_readlane(n, l),
                h0};
  }
  return Span{-1, 0, 0, 0, 0, 0};
}

// Slots of all groups.
__device__ __forceinline__ int32_t total_slots(const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                               uint32_t unit) {
  if (groups == 0) return int32_t((uint32_t(rows) + unit - 1) / unit);
  int32_t carry = clamp_row(offsets[0], rows), base = 0;
  for (int32_t e0 = 0; e0 < groups; e0 += 64) {
    int32_t lo, hi, first, n;
    group_block(offsets, groups, rows, unit, e0, carry, base, lo, hi, first, n);
  }
  return base;
}

// All rows and the slots of group e.
__device__ __forceinline__ Span group_span(const int64_t* __restrict__ offsets, int32_t groups, int32_t rows,
                                           uint32_t unit, int32_t e) {
  if (groups == 0) return Span{0, 0, rows, 0, int32_t((uint32_t(rows) + unit - 1) / unit), rows};
  int32_t carry = clamp_row(offsets[0], rows), base = 0;
  for (int32_t e0 = 0;; e0 += 64) {
    int32_t lo, hi, first, n;
    group_block(offsets, groups, rows, unit, e0, carry, base, lo, hi, first, n);
    if (e >= e0 + 64) continue;
    const int l = e - e0;
    return Span{e, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(hi, l),
                __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(n, l),
                __builtin_amdgcn_readlane(hi, l)};
  }
}

// Lanes of a wave exchange data through LDS that is the wave's own: orders
// the accesses before against those after, without a workgroup barrier.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace net
}  // namespace gs
