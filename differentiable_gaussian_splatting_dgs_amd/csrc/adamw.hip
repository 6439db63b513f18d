// One AdamW step over many tensors in one launch.
//
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps),  c = 1 - b^t
//
// Bound by the bytes: p, m and v in and out, g in, the copy out.  The tensors'
// addresses travel as the launch's arguments; a workgroup finds its tensor by
// bisection of their first workgroups and works on kGroup of its elements.
//
// Moments in 8 bits share a power of two for each 256 values, which are the
// four neighbours of each lane of a wave: the largest magnitude is one wave
// maximum, and the scale comes out as a scalar.  A code is decided by where
// its value lies between two steps, so the new moments are worked out in 64
// bits, for which a pass that is bound by memory has room (10 instructions a
// value); rounding needs no more than the upper word of a value:
//   - its 20 bits behind the point are the 3 of the code and 17 of what is
//     rounded away;
//   - adding a number below 2^17 and cutting off rounds up with the
//     probability of what is cut off.  The number is odd (2 u + 1, u of 16
//     bits), so that the cut off low word cannot decide.
// p's square root and reciprocal are the hardware's (about 1 ulp each, far
// below the rounding that p's own sum makes of a small update).
#include <algorithm>
#include <cmath>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                          // quads of a thread
constexpr int kGroup = kThreads * 4 * kUnroll;      // elements of a workgroup

struct AdamwBatch {
  AdamwTensor t[kAdamwTensors];
  int32_t count;
};
struct AdamwNumbers {
  double b1, ob1, b2, ob2;      // 1 - beta in 64 bits
  double log_b1, log_b2;
  double lr;
  float decay, eps;
  float rate, inv_c2;           // lr / c1, 1 / c2 where the step is known
  uint32_t step;
  const int64_t* step_dev;
  const float* grad_scale;
};
static_assert(sizeof(AdamwBatch) + sizeof(AdamwNumbers) <= 4096, "kernel arguments");

// 32 bits mixed: each bit of the result depends on all of x.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;
  x ^= x >> 15;
  x *= 0xB7E15163u;
  return x ^ (x >> 16);
}

// Four neighbours; n of them exist.
__device__ __forceinline__ void load4(const float* __restrict__ p, int n, float (&v)[4]) {
  const Chunk<float> c = load_chunk_n(p, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = c.v[i];
}
__device__ __forceinline__ void store4(float* __restrict__ p, int n, const float (&v)[4]) {
  Chunk<float> c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = v[i];
  store_chunk_n(p, c, n);
}
template <typename T>
__device__ __forceinline__ void load4_half(const T* __restrict__ p, int n, float (&v)[4]) {
  T c[4] = {};
  if (n >= 4)
    __builtin_memcpy(c, p, 8);
  else
    for (int i = 0; i < n; ++i) c[i] = p[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float(c[i]);
}
template <typename T>
__device__ __forceinline__ void store4_half(T* __restrict__ p, int n, const float (&v)[4]) {
  T c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = T(v[i]);
  if (n >= 4)
    __builtin_memcpy(p, c, 8);
  else
    for (int i = 0; i < n; ++i) p[i] = c[i];
}
__device__ __forceinline__ void load4_typed(const void* __restrict__ p, int type, int64_t at, int n, float (&v)[4]) {
  if (type == kTypeF32)
    load4(static_cast<const float*>(p) + at, n, v);
  else if (type == kTypeBF16)
    load4_half(static_cast<const bf16*>(p) + at, n, v);
  else
    load4_half(static_cast<const f16*>(p) + at, n, v);
}
__device__ __forceinline__ void store4_typed(void* __restrict__ p, int type, int64_t at, int n, const float (&v)[4]) {
  if (type == kTypeF32)
    store4(static_cast<float*>(p) + at, n, v);
  else if (type == kTypeBF16)
    store4_half(static_cast<bf16*>(p) + at, n, v);
  else
    store4_half(static_cast<f16*>(p) + at, n, v);
}
__device__ __forceinline__ uint32_t load4_codes(const uint8_t* __restrict__ p, int n) {
  uint32_t c = 0;
  if (n >= 4)
    __builtin_memcpy(&c, p, 4);
  else
    for (int i = 0; i < n; ++i) c |= uint32_t(p[i]) << (8 * i);
  return c;
}
__device__ __forceinline__ void store4_codes(uint8_t* __restrict__ p, int n, uint32_t c) {
  if (n >= 4)
    __builtin_memcpy(p, &c, 4);
  else
    for (int i = 0; i < n; ++i) p[i] = uint8_t(c >> (8 * i));
}

// --- codes -----------------------------------------------------------------------

// With its 5 or 4 bits e and 3 bits f as the exponent's and the first bits of a
// float, a code is that float's value times 2^129, for e = 0 (subnormal) too.
__device__ __forceinline__ float code_size(uint32_t c) {
  return ldexpf(__builtin_bit_cast(float, c << 20), 129);
}
template <bool kSigned>
__device__ __forceinline__ float decode(uint32_t c, float scale) {
  if constexpr (kSigned) {
    const float x = code_size(c & 127u) * scale;
    return (c & 127u) == 127u ? __builtin_nanf("") : (c & 128u) != 0 ? -x : x;
  } else {
    return c == 255u ? __builtin_nanf("") : code_size(c) * scale;
  }
}

// A value's upper word without its sign; 0 for one that does not count
// towards the block's largest.
__device__ __forceinline__ uint32_t upper(double x) {
  return uint32_t(__builtin_bit_cast(uint64_t, x) >> 32) & 0x7FFFFFFFu;
}

// The largest of a wave's words, a scalar.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define GS_DPP_MAX(ctrl, rows)                                                                        \
  {                                                                                                   \
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), ctrl, rows, 0xF, false));      \
    v = v > o ? v : o;                                                                                \
  }
  GS_DPP_MAX(0xB1, 0xF)    // quad_perm 1 0 3 2
  GS_DPP_MAX(0x4E, 0xF)    // quad_perm 2 3 0 1
  GS_DPP_MAX(0x141, 0xF)   // half mirror
  GS_DPP_MAX(0x140, 0xF)   // mirror
  GS_DPP_MAX(0x142, 0xA)   // lane 15 to the row after, rows 1 and 3
  GS_DPP_MAX(0x143, 0xC)   // lane 31 to rows 2 and 3
#undef GS_DPP_MAX
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// Exponent of the scale under which `most` is at most 14 steps of the last
// octave (of kOctaves; 15 with a carry would be NaN's code).
template <int kOctaves>
__device__ __forceinline__ int unit_of(uint32_t most) {
  const int e = int(most >> 20) - 1023 + ((most & 0xFFFFFu) >= 0xC0000u ? 1 : 0);
  const int unit = e - 3 - (kOctaves - 1);
  return unit < -126 ? -126 : unit;
}

__device__ __forceinline__ uint32_t encode(uint32_t word, int unit, uint32_t odd) {
  const int above = int(word >> 20) - 1023 - 3 - unit;      // octaves over the first
  const int down = above < 0 ? -above : 0;
  const uint32_t steps = (((word & 0xFFFFFu) | 0x100000u) >> (down < 31 ? down : 31)) + odd;
  return (steps >> 17) + 8u * uint32_t(above > 0 ? above : 0);
}

// --- the step ----------------------------------------------------------------------

struct StepNumbers {
  float rate, inv_c2, scale;
  uint32_t step;
};
__device__ __forceinline__ StepNumbers step_numbers(const AdamwNumbers& h) {
  StepNumbers s{h.rate, h.inv_c2, 1.0f, h.step};
  if (h.step_dev != nullptr) {
    const int64_t t = std::max<int64_t>(*h.step_dev, 1);
    s.rate = float(h.lr / -expm1(double(t) * h.log_b1));
    s.inv_c2 = float(1.0 / -expm1(double(t) * h.log_b2));
    s.step = uint32_t(t);
  }
  if (h.grad_scale != nullptr) s.scale = *h.grad_scale;
  return s;
}

__device__ __forceinline__ int tensor_of(const AdamwBatch& b) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].first <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float update(float p, float m, float v, const AdamwNumbers& h, const StepNumbers& s) {
  const float d = __builtin_amdgcn_sqrtf(v * s.inv_c2) + h.eps;
  return fmaf(p, h.decay, -(s.rate * m * __builtin_amdgcn_rcpf(d)));
}

__global__ __launch_bounds__(kThreads) void k_adamw(AdamwBatch b, AdamwNumbers h) {
  const AdamwTensor& t = b.t[tensor_of(b)];
  const StepNumbers s = step_numbers(h);
  const float b1 = float(h.b1), ob1 = float(h.ob1), b2 = float(h.b2), ob2 = float(h.ob2);
  const int64_t base = int64_t(blockIdx.x - t.first) * kGroup;
  float *const m = static_cast<float*>(t.m), *const v = static_cast<float*>(t.v);
  float vp[kUnroll][4], vg[kUnroll][4], vm[kUnroll][4], vv[kUnroll][4];
  int n[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = base + (u * kThreads + threadIdx.x) * 4;
    n[u] = int(std::min<int64_t>(4, std::max<int64_t>(0, t.n - at)));
    load4(t.param + at, n[u], vp[u]);
    load4_typed(t.grad, t.grad_type, at, n[u], vg[u]);
    load4(m + at, n[u], vm[u]);
    load4(v + at, n[u], vv[u]);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = base + (u * kThreads + threadIdx.x) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g = vg[u][i] * s.scale;
      vm[u][i] = fmaf(b1, vm[u][i], ob1 * g);
      vv[u][i] = fmaf(b2, vv[u][i], ob2 * (g * g));
      vp[u][i] = update(vp[u][i], vm[u][i], vv[u][i], h, s);
    }
    store4(t.param + at, n[u], vp[u]);
    store4(m + at, n[u], vm[u]);
    store4(v + at, n[u], vv[u]);
    if (t.copy != nullptr) store4_typed(t.copy, t.copy_type, at, n[u], vp[u]);
  }
}

__global__ __launch_bounds__(kThreads) void k_adamw_8(AdamwBatch b, AdamwNumbers h) {
  const AdamwTensor& t = b.t[tensor_of(b)];
  const StepNumbers s = step_numbers(h);
  const uint32_t key = mix(t.key + s.step);
  const int64_t base = int64_t(blockIdx.x - t.first) * kGroup;
  uint8_t *const m = static_cast<uint8_t*>(t.m), *const v = static_cast<uint8_t*>(t.v);
  float vp[kUnroll][4], vg[kUnroll][4], ms[kUnroll], vs[kUnroll];
  uint32_t cm[kUnroll], cv[kUnroll];
  int n[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = base + (u * kThreads + threadIdx.x) * 4;
    n[u] = int(std::min<int64_t>(4, std::max<int64_t>(0, t.n - at)));
    load4(t.param + at, n[u], vp[u]);
    load4_typed(t.grad, t.grad_type, at, n[u], vg[u]);
    cm[u] = load4_codes(m + at, n[u]);
    cv[u] = load4_codes(v + at, n[u]);
    ms[u] = n[u] > 0 ? t.m_scale[at / kAdamwBlock] : 0.0f;
    vs[u] = n[u] > 0 ? t.v_scale[at / kAdamwBlock] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = base + (u * kThreads + threadIdx.x) * 4;
    uint32_t wm[4], wv[4], signs = 0, most_m = 0, most_v = 0;
    uint32_t lost = 0, some = 0;      // bits: not finite; v over 0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double g = double(vg[u][i]) * double(s.scale);
      const double m1 = fma(h.b1, double(decode<true>((cm[u] >> (8 * i)) & 255u, ms[u])), h.ob1 * g);
      const double v1 = fma(h.b2, double(decode<false>((cv[u] >> (8 * i)) & 255u, vs[u])), h.ob2 * (g * g));
      const float mf = float(m1), vf = float(v1);
      const bool bad_m = !__builtin_isfinite(mf), bad_v = !__builtin_isfinite(vf);
      wm[i] = bad_m ? 0u : upper(m1);
      wv[i] = bad_v ? 0u : upper(v1);
      lost |= (bad_m ? 1u : 0u) << i | (bad_v ? 16u : 0u) << i;
      some |= (v1 > 0.0 ? 1u : 0u) << i;
      signs |= (m1 < 0.0 ? 128u : 0u) << (8 * i);
      most_m = most_m > wm[i] ? most_m : wm[i];
      most_v = most_v > wv[i] ? most_v : wv[i];
      vp[u][i] = update(vp[u][i], mf, vf, h, s);
    }
    const int unit_m = unit_of<15>(wave_max(most_m)), unit_v = unit_of<31>(wave_max(most_v));
    uint32_t out_m = 0, out_v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t e = uint64_t(at) + i;
      const uint32_t random = mix(uint32_t(e) ^ (uint32_t(e >> 32) * 0x9E3779B9u) ^ key);
      uint32_t c = encode(wm[i], unit_m, (random & 0xFFFFu) * 2 + 1);
      c = (lost >> i & 1u) != 0 ? 127u : c;
      out_m |= c << (8 * i);
      c = encode(wv[i], unit_v, (random >> 16) * 2 + 1);
      c = c == 0 ? some >> i & 1u : c;
      c = (lost >> i & 16u) != 0 ? 255u : c;
      out_v |= c << (8 * i);
    }
    if (n[u] > 0) {
      store4(t.param + at, n[u], vp[u]);
      store4_codes(m + at, n[u], out_m | signs);
      store4_codes(v + at, n[u], out_v);
      if ((threadIdx.x & 63) == 0) {
        t.m_scale[at / kAdamwBlock] = __builtin_bit_cast(float, uint32_t(unit_m + 127) << 23);
        t.v_scale[at / kAdamwBlock] = __builtin_bit_cast(float, uint32_t(unit_v + 127) << 23);
      }
      if (t.copy != nullptr) store4_typed(t.copy, t.copy_type, at, n[u], vp[u]);
    }
  }
}

template <bool kSigned>
__global__ __launch_bounds__(kThreads) void k_moment(const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scales, int64_t n, int type,
                                                     void* __restrict__ values) {
  for (int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 4; at < n; at += int64_t(gridDim.x) * kThreads * 4) {
    const int k = int(std::min<int64_t>(4, n - at));
    const uint32_t c = load4_codes(codes + at, k);
    const float scale = scales[at / kAdamwBlock];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = decode<kSigned>((c >> (8 * i)) & 255u, scale);
    store4_typed(values, type, at, k, v);
  }
}

}  // namespace
}  // namespace net

uint32_t adamw_key(uint64_t seed, uint32_t place) {
  return net::mix(net::mix(uint32_t(seed) ^ place) + uint32_t(seed >> 32));
}

uint32_t adamw_workgroups(int64_t n) { return uint32_t((n + net::kGroup - 1) / net::kGroup); }

hipError_t launch_adamw(const AdamwTensor* tensors, int count, bool eight, uint32_t workgroups, const AdamwHyper& h,
                        hipStream_t st) {
  net::AdamwBatch b;
  std::copy(tensors, tensors + count, b.t);
  b.count = count;
  net::AdamwNumbers k{};
  k.b1 = h.beta1;
  k.ob1 = 1.0 - h.beta1;
  k.b2 = h.beta2;
  k.ob2 = 1.0 - h.beta2;
  k.log_b1 = std::log(h.beta1);
  k.log_b2 = std::log(h.beta2);
  k.lr = h.lr;
  k.decay = float(1.0 - h.lr * h.weight_decay);
  k.eps = float(h.eps);
  k.step_dev = h.step_dev;
  k.grad_scale = h.grad_scale;
  if (h.step_dev == nullptr) {
    k.rate = float(h.lr / -std::expm1(double(h.step) * k.log_b1));
    k.inv_c2 = float(1.0 / -std::expm1(double(h.step) * k.log_b2));
    k.step = uint32_t(h.step);
  }
  if (eight)
    net::k_adamw_8<<<workgroups, net::kThreads, 0, st>>>(b, k);
  else
    net::k_adamw<<<workgroups, net::kThreads, 0, st>>>(b, k);
  return hipGetLastError();
}

hipError_t launch_adamw_moment(const uint8_t* codes, const float* scales, int64_t n, int moment, int type,
                               void* values, hipStream_t st) {
  const unsigned grid = net::grid_of((n + net::kThreads * 4 - 1) / (net::kThreads * 4));
  if (moment == 1)
    net::k_moment<true><<<grid, net::kThreads, 0, st>>>(codes, scales, n, type, values);
  else
    net::k_moment<false><<<grid, net::kThreads, 0, st>>>(codes, scales, n, type, values);
  return hipGetLastError();
}

}  // namespace gs
