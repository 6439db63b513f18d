// One AdamW step over many tensors in one launch.
//
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps),  c = 1 - b^t
//
// Bound by the bytes: p, m and v in and out, g in, the copy out.  The nine
// tensors of a decoder with 500,003 x 64 features, fp32: 176 us (963 MB at 5.5
// TB/s); 1,000,003 x 64, bf16 gradients, moments in 8 bits: 192 to 215 us (1.04 GB
// at 4.8 to 5.4 TB/s, 70 vector instructions a value).  A step whose number is on
// the device works out its corrections in every thread: 8 and 18 us more with
// the launch that counts.  The tensors'
// addresses travel as the launch's arguments; a workgroup finds its tensor by
// bisection of their first workgroups and works on kGroup of its elements.
//
// Moments in 8 bits share a power of two for each 256 values, which are the
// four neighbours of each lane of a wave: the largest magnitude is one wave
// maximum, and the scale comes out as a scalar.  A code is decided by where
// its value lies between two steps, so the new moments are worked out in 64
// bits; rounding needs no more than the upper word of a value:
//   - its 20 bits behind the point are the 3 of the code and 17 of what is
//     rounded away;
//   - adding a number below 2^17 and cutting off rounds up with the
//     probability of what is cut off.  The number is odd (2 u + 1, u of 16
//     bits), so that the cut off low word cannot decide.
// What only few blocks need (values below the scale's first octave, infinities
// and NaN) is behind branches that a whole wave takes or not: every instruction
// for each value counts, the vector unit is about as long as the memory.
// p's square root and reciprocal are the hardware's (about 1 ulp each, far
// below the rounding that p's own sum makes of a small update), which take
// subnormal numbers as 0: where eps is that small, the update scales them.
#include <algorithm>
#include <cmath>

#include "row_chunks.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;
// Elements of a workgroup: four a thread, so that a wave's registers leave room
// for more waves (calls in a row as it was chosen, 500,003 x 64 fp32: 179 us, with
// 8 a thread 183, 16 186; 8 bits with the moments read out: 328, 339, 349).
constexpr int kGroup = kThreads * 4;

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

// Four neighbours at p; n of them exist.
template <typename T>
__device__ __forceinline__ void load4(const T* __restrict__ p, int n, float (&v)[4]) {
  T c[4] = {};
  if (n == 4) {
    __builtin_memcpy(c, p, sizeof(c));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) c[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float(c[i]);
}
template <typename T>
__device__ __forceinline__ void store4(T* __restrict__ p, int n, const float (&v)[4]) {
  T c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = T(v[i]);
  if (n == 4) {
    __builtin_memcpy(p, c, sizeof(c));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) p[i] = c[i];
  }
}
__device__ __forceinline__ void store4_typed(void* __restrict__ p, int type, int64_t at, int n, const float (&v)[4]) {
  if (type == kTypeF32)
    store4(static_cast<float*>(p) + at, n, v);
  else if (type == kTypeBF16)
    store4(static_cast<bf16*>(p) + at, n, v);
  else
    store4(static_cast<f16*>(p) + at, n, v);
}
__device__ __forceinline__ uint32_t load4_codes(const uint8_t* __restrict__ p, int n) {
  uint32_t c = 0;
  if (n == 4)
    __builtin_memcpy(&c, p, 4);
  else
    for (int i = 0; i < n; ++i) c |= uint32_t(p[i]) << (8 * i);
  return c;
}
__device__ __forceinline__ void store4_codes(uint8_t* __restrict__ p, int n, uint32_t c) {
  if (n == 4)
    __builtin_memcpy(p, &c, 4);
  else
    for (int i = 0; i < n; ++i) p[i] = uint8_t(c >> (8 * i));
}

// --- codes -----------------------------------------------------------------------

// With its 5 bits e and 3 bits f as the last of the exponent's and the first of
// the fraction's, a code is that float's value times 2^129, for e = 0 (subnormal)
// too.  m's codes are the 8-bit floats e4m3fn, with a factor of 2^9.
__device__ __forceinline__ float code_bits(uint32_t codes, int i) {
  return __builtin_bit_cast(float, (i == 3 ? codes >> 4 : codes << (20 - 8 * i)) & 0x0FF00000u);
}
constexpr double kCodeV = 0x1p129, kCodeM = 512.0;
__device__ __forceinline__ bool is_lost(uint32_t codes, int i) { return ((codes >> (8 * i)) & 255u) == 255u; }
// Whether one of four v's is NaN's code.
__device__ __forceinline__ bool any_lost(uint32_t codes) {
  return ((codes & 0x7F7F7F7Fu) + 0x01010101u & codes & 0x80808080u) != 0;
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void floats_of(uint32_t codes, float (&v)[4]) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(codes), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(codes), true);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// A value's upper word without its sign, and that of 2^128.
__device__ __forceinline__ uint32_t upper(double x) {
  return uint32_t(__builtin_bit_cast(uint64_t, x) >> 32);
}
constexpr uint32_t kTooLarge = 0x47F00000u;

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

// Exponent of the scale under which `most` is below 14 steps of the last octave
// (of kOctaves): from 14 and a part of one on it may be rounded to 15, NaN's
// code, and the word's cut off half does not tell 14 from that.
template <int kOctaves>
__device__ __forceinline__ int unit_of(uint32_t most) {
  const int e = int(most >> 20) - 1023 + ((most & 0xFFFFFu) >= 0xC0000u ? 1 : 0);
  const int unit = e - 3 - (kOctaves - 1);
  return unit < -126 ? -126 : unit;
}

// Codes of four upper words under a scale of 2^unit: the word, with the random
// number added behind its first three bits of fraction, less the exponent of
// the first octave; a value below that octave has its fraction shifted.
__device__ __forceinline__ void encode4(const uint32_t (&word)[4], int unit, const uint32_t (&odd)[4],
                                        uint32_t (&code)[4]) {
  const uint32_t first = uint32_t(unit + 3 + 1023) << 20;
  uint32_t least = word[0] < word[1] ? word[0] : word[1];
  least = least < word[2] ? least : word[2];
  least = least < word[3] ? least : word[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = ((word[i] + odd[i]) >> 17) - ((first >> 17) - 8u);
  if (__builtin_amdgcn_ballot_w64(least < first) != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t down = (first >> 20) - (word[i] >> 20);
      const uint32_t steps = (((word[i] & 0xFFFFFu) | 0x100000u) >> (down < 31u ? down : 31u)) + odd[i];
      code[i] = word[i] < first ? steps >> 17 : code[i];
    }
  }
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

// The root of a subnormal number is under 2^-63: taken as 0 it is at most half
// a step of an eps from 2^-39 on.  A smaller eps (the same branch for all):
// where the root is under k^-1 = 2^-32, root and eps are taken k times and,
// so that its product with the rate is no subnormal, a small m is too.  eps is
// at least 2^-126 and at most 2^125, so that no reciprocal leaves fp32.
constexpr float kPlainEps = 0x1p-39f;
__device__ __forceinline__ float update(float p, float m, float v, const AdamwNumbers& h, const StepNumbers& s) {
  const float x = v * s.inv_c2;
  float step;
  if (h.eps >= kPlainEps) {
    step = s.rate * m * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(x) + h.eps);
  } else {
    const float k = x < 0x1p-64f ? 0x1p32f : 1.0f;
    const float r = __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(x * k * k) + h.eps * k);
    const bool small = fabsf(m) < 0x1p-32f;
    step = s.rate * (small ? m * k : m) * (small ? r : r * k);
  }
  return fmaf(p, h.decay, -step);
}

// G: the gradients' type.
template <typename G>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamwBatch b, AdamwNumbers h) {
  const AdamwTensor& t = b.t[tensor_of(b)];
  const StepNumbers s = step_numbers(h);
  const float b1 = float(h.b1), ob1 = float(h.ob1), b2 = float(h.b2), ob2 = float(h.ob2);
  const int64_t at = int64_t(blockIdx.x - t.first) * kGroup + threadIdx.x * 4;
  if (at >= t.n) return;
  const int n = int(std::min<int64_t>(4, t.n - at));
  float p[4], g[4], m[4], v[4];
  load4(t.param + at, n, p);
  load4(static_cast<const float*>(t.m) + at, n, m);
  load4(static_cast<const float*>(t.v) + at, n, v);
  load4(static_cast<const G*>(t.grad) + at, n, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] *= s.scale;
    m[i] = fmaf(b1, m[i], ob1 * g[i]);
    v[i] = fmaf(b2, v[i], ob2 * (g[i] * g[i]));
    p[i] = update(p[i], m[i], v[i], h, s);
  }
  store4(t.param + at, n, p);
  store4(static_cast<float*>(t.m) + at, n, m);
  store4(static_cast<float*>(t.v) + at, n, v);
  if (t.copy != nullptr) store4_typed(t.copy, t.copy_type, at, n, p);
}

template <typename G>
__global__ __launch_bounds__(kThreads) void k_adamw_8(AdamwBatch b, AdamwNumbers h) {
  const AdamwTensor& t = b.t[tensor_of(b)];
  const StepNumbers s = step_numbers(h);
  const uint32_t key = mix(t.key + s.step);
  // a wave has one block, the last one's behind the tensor's end included
  const int64_t at = int64_t(blockIdx.x - t.first) * kGroup + threadIdx.x * 4, block = at / kAdamwBlock;
  if (block * kAdamwBlock >= t.n) return;
  const int n = int(std::min<int64_t>(4, std::max<int64_t>(0, t.n - at)));
  float p[4], g[4], m0[4];
  load4(t.param + at, n, p);
  load4(static_cast<const G*>(t.grad) + at, n, g);
  const uint32_t cm = load4_codes(static_cast<const uint8_t*>(t.m) + at, n);
  const uint32_t cv = load4_codes(static_cast<const uint8_t*>(t.v) + at, n);
  const double b1 = h.b1 * kCodeM * double(t.m_scale[block]), b2 = h.b2 * kCodeV * double(t.v_scale[block]);
  const double ob1 = h.ob1 * double(s.scale), ob2 = h.ob2 * double(s.scale) * double(s.scale);
  floats_of(cm, m0);
  double m1[4], v1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double x = double(g[i]);
    m1[i] = fma(b1, double(m0[i]), ob1 * x);
    v1[i] = fma(ob2, x * x, b2 * double(code_bits(cv, i)));
  }
  if (__builtin_amdgcn_ballot_w64(any_lost(cv)) != 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) v1[i] = is_lost(cv, i) ? __builtin_nan("") : v1[i];
  uint32_t wm[4], wv[4], most_m = 0, most_v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = update(p[i], float(m1[i]), float(v1[i]), h, s);
    wm[i] = upper(m1[i]) & 0x7FFFFFFFu;
    wv[i] = upper(v1[i]) & 0x7FFFFFFFu;
    most_m = most_m > wm[i] ? most_m : wm[i];
    most_v = most_v > wv[i] ? most_v : wv[i];
  }
  most_m = wave_max(most_m);
  most_v = wave_max(most_v);
  uint32_t lost = 0;      // bits of values that are not finite, which do not count for the scale
  if (most_m >= kTooLarge || most_v >= kTooLarge) {
    most_m = most_v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lost |= (wm[i] >= kTooLarge ? 1u : 0u) << i | (wv[i] >= kTooLarge ? 16u : 0u) << i;
      wm[i] = wm[i] >= kTooLarge ? 0u : wm[i];
      wv[i] = wv[i] >= kTooLarge ? 0u : wv[i];
      most_m = most_m > wm[i] ? most_m : wm[i];
      most_v = most_v > wv[i] ? most_v : wv[i];
    }
    most_m = wave_max(most_m);
    most_v = wave_max(most_v);
  }
  const int unit_m = unit_of<15>(most_m), unit_v = unit_of<31>(most_v);
  uint32_t odd_m[4], odd_v[4], c_m[4], c_v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t e = uint64_t(at) + i;
    const uint32_t random = mix(uint32_t(e) ^ uint32_t(uint64_t(at) >> 32) * 0x9E3779B9u ^ key);
    odd_m[i] = (random & 0xFFFFu) * 2 + 1;
    odd_v[i] = random >> 15 | 1u;
  }
  encode4(wm, unit_m, odd_m, c_m);
  encode4(wv, unit_v, odd_v, c_v);
  uint32_t out_m = 0, out_v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c_m[i] |= upper(m1[i]) >> 24 & 128u;
    const uint32_t some = wv[i] < 1u ? wv[i] : 1u;
    out_m |= c_m[i] << (8 * i);
    out_v |= (c_v[i] > some ? c_v[i] : some) << (8 * i);
  }
  if (__builtin_amdgcn_ballot_w64(lost != 0) != 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((lost >> i & 1u) != 0) out_m |= 127u << (8 * i);
      if ((lost >> i & 16u) != 0) out_v |= 255u << (8 * i);
    }
  if (n > 0) {
    store4(t.param + at, n, p);
    store4_codes(static_cast<uint8_t*>(t.m) + at, n, out_m);
    store4_codes(static_cast<uint8_t*>(t.v) + at, n, out_v);
    if (t.copy != nullptr) store4_typed(t.copy, t.copy_type, at, n, p);
    if ((threadIdx.x & 63) == 0) {
      t.m_scale[block] = __builtin_bit_cast(float, uint32_t(unit_m + 127) << 23);
      t.v_scale[block] = __builtin_bit_cast(float, uint32_t(unit_v + 127) << 23);
    }
  }
}

constexpr int kMomentAhead = 4;

template <typename T, bool kSigned>
__device__ __forceinline__ void values_of(uint32_t codes, float scale, T* __restrict__ out) {
  float v[4];
  if constexpr (kSigned) {
    floats_of(codes, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = T(v[i] * float(kCodeM) * scale);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out[i] = T(is_lost(codes, i) ? __builtin_nanf("") : ldexpf(code_bits(codes, i), 129) * scale);
  }
}

// kMomentAhead stores of 16 bytes a thread, neighbours by neighbouring lanes;
// the tensor's last elements one by one.
template <typename T, bool kSigned>
__global__ __launch_bounds__(kThreads) void k_moment(const uint8_t* __restrict__ codes,
                                                     const float* __restrict__ scales, int64_t n,
                                                     T* __restrict__ values) {
  constexpr int K = kChunk<T>, kStep = kThreads * K;
  for (int64_t first = int64_t(blockIdx.x) * kStep * kMomentAhead; first < n;
       first += int64_t(gridDim.x) * kStep * kMomentAhead) {
    if (first + kStep * kMomentAhead > n) {      // the same for the whole workgroup
      for (int64_t at = first + threadIdx.x; at < n; at += kThreads) {
        T v[4];
        values_of<T, kSigned>(codes[at], scales[at / kAdamwBlock], v);
        values[at] = v[0];
      }
      return;
    }
    const int64_t base = first + threadIdx.x * K;
    uint32_t word[kMomentAhead][K / 4];
    float scale[kMomentAhead];
#pragma unroll
    for (int u = 0; u < kMomentAhead; ++u) {
      __builtin_memcpy(word[u], codes + base + u * kStep, K);
      scale[u] = scales[(base + u * kStep) / kAdamwBlock];
    }
#pragma unroll
    for (int u = 0; u < kMomentAhead; ++u) {
      Chunk<T> o;
#pragma unroll
      for (int q = 0; q < K; q += 4) values_of<T, kSigned>(word[u][q / 4], scale[u], o.v + q);
      store_chunk(values + base + u * kStep, o);
    }
  }
}

template <typename T>
void go_moment(const uint8_t* codes, const float* scales, int64_t n, int moment, void* values, hipStream_t st) {
  constexpr int64_t kEach = int64_t(kThreads) * kChunk<T> * kMomentAhead;
  const unsigned grid = grid_of((n + kEach - 1) / kEach);
  if (moment == 1)
    k_moment<T, true><<<grid, kThreads, 0, st>>>(codes, scales, n, static_cast<T*>(values));
  else
    k_moment<T, false><<<grid, kThreads, 0, st>>>(codes, scales, n, static_cast<T*>(values));
}

template <typename G>
void go(bool eight, uint32_t workgroups, const AdamwBatch& b, const AdamwNumbers& k, hipStream_t st) {
  if (eight)
    k_adamw_8<G><<<workgroups, kThreads, 0, st>>>(b, k);
  else
    k_adamw<G><<<workgroups, kThreads, 0, st>>>(b, k);
}

}  // namespace
}  // namespace net

uint32_t adamw_key(uint64_t seed, uint32_t place) {
  return net::mix(net::mix(uint32_t(seed) ^ place) + uint32_t(seed >> 32));
}

uint32_t adamw_workgroups(int64_t n) { return uint32_t((n + net::kGroup - 1) / net::kGroup); }

hipError_t launch_adamw(const AdamwTensor* tensors, int count, bool eight, int grad_type, uint32_t workgroups,
                        const AdamwHyper& h, hipStream_t st) {
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
  if (grad_type == kTypeF32)
    net::go<float>(eight, workgroups, b, k, st);
  else if (grad_type == kTypeBF16)
    net::go<net::bf16>(eight, workgroups, b, k, st);
  else
    net::go<net::f16>(eight, workgroups, b, k, st);
  return hipGetLastError();
}

hipError_t launch_adamw_moment(const uint8_t* codes, const float* scales, int64_t n, int moment, int type,
                               void* values, hipStream_t st) {
  if (type == kTypeF32)
    net::go_moment<float>(codes, scales, n, moment, values, st);
  else if (type == kTypeBF16)
    net::go_moment<net::bf16>(codes, scales, n, moment, values, st);
  else
    net::go_moment<net::f16>(codes, scales, n, moment, values, st);
  return hipGetLastError();
}

}  // namespace gs
