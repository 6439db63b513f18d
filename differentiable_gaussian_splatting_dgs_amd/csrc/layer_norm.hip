// Layer norm over the last axis, forward and backward, with the reduction of
// the weights' gradients.
//
//   forward   mean = sum x / d, var = sum (x - mean)^2 / d (both passes over
//             the row held in registers), rstd = 1 / sqrt(var + eps),
//             y = gamma (x - mean) rstd + beta
//   backward  xh = (x - mean) rstd, g = dy gamma,
//             dx = rstd (g - mean(g) - xh mean(g xh)) (+ dres),
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//
// Bound by HBM: each row is read once and written once.  A row is held by L
// lanes of C 16-byte chunks each, so a wave works on 64 / L rows and its
// loads are contiguous.  Statistics and sums are fp32; the only rounding to
// fewer bits is the one of y and dx into their storage.
#include <algorithm>

#include "net_common.hpp"

namespace gs {
namespace net {
namespace {

constexpr int kThreads = 256;
// Workgroups of the backward pass: each leaves one partial row of dgamma
// and dbeta, so their number is also the length of the second reduction.
constexpr int kBwdGroups = 1024;
constexpr int kFwdGroups = 2048;

// Sum over the L lanes of a row (L <= 64: lanes of one wave; L = 256: the
// workgroup), the same on all of them.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* s) {
#pragma unroll
  for (int d = 1; d < (L < 64 ? L : 64); d <<= 1) v += __shfl_xor(v, d, 64);
  if constexpr (L > 64) {
    __syncthreads();   // the previous sum's readers are done
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (s[0] + s[1]) + (s[2] + s[3]);
  }
  return v;
}

template <typename T, int L, int C>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(NormArgs a) {
  constexpr int K = kChunk<T>, kRows = kThreads / L;
  __shared__ float s[4];
  const int l = threadIdx.x % L, d = a.width;
  const T* __restrict__ x = static_cast<const T*>(a.x);
  T* __restrict__ y = static_cast<T*>(a.y);
  float gm[C][K], bt[C][K];
  int n[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c0 = (l + L * j) * K;
    n[j] = std::min(K, std::max(0, d - c0));
#pragma unroll
    for (int i = 0; i < K; ++i) {
      gm[j][i] = a.gamma != nullptr && i < n[j] ? a.gamma[c0 + i] : 1.0f;
      bt[j][i] = a.beta != nullptr && i < n[j] ? a.beta[c0 + i] : 0.0f;
    }
  }
  const float inv_d = 1.0f / float(d);
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < a.rows; r0 += int64_t(gridDim.x) * kRows) {
    const int64_t r = r0 + threadIdx.x / L;
    const bool live = r < a.rows;
    float v[C][K];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const Chunk<T> c = load_chunk_n(x + r * a.ldx + (l + L * j) * K, live ? n[j] : 0);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        v[j][i] = float(c.v[i]);
        sum += v[j][i];
      }
    }
    const float mean = row_sum<L>(sum, s) * inv_d;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < K; ++i) {
        v[j][i] = i < n[j] ? v[j][i] - mean : 0.0f;
        sq = fmaf(v[j][i], v[j][i], sq);
      }
    const float rstd = 1.0f / sqrtf(row_sum<L>(sq, s) * inv_d + a.eps);
    if (!live) continue;   // L = 256 has one row, so the workgroup stays together
    if (l == 0) {
      if (a.mean != nullptr) a.mean[r] = mean;
      if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (n[j] == 0) continue;
      Chunk<T> c;
#pragma unroll
      for (int i = 0; i < K; ++i) c.v[i] = T(fmaf(v[j][i] * rstd, gm[j][i], bt[j][i]));
      store_chunk_n(y + r * a.ldy + (l + L * j) * K, c, n[j]);
    }
  }
}

// dx of its rows and one partial row of dgamma and dbeta: part[workgroup][2][d].
template <typename T, int L, int C>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(NormArgs a, float* __restrict__ part) {
  constexpr int K = kChunk<T>, kRows = kThreads / L;
  __shared__ float s[4];
  const int l = threadIdx.x % L, d = a.width;
  const T* __restrict__ x = static_cast<const T*>(a.x);
  const T* __restrict__ dy = static_cast<const T*>(a.dy);
  const T* __restrict__ dres = static_cast<const T*>(a.dres);
  T* __restrict__ dx = static_cast<T*>(a.dx);
  float gm[C][K], ag[C][K], ab[C][K];
  int n[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c0 = (l + L * j) * K;
    n[j] = std::min(K, std::max(0, d - c0));
#pragma unroll
    for (int i = 0; i < K; ++i) {
      gm[j][i] = a.gamma != nullptr && i < n[j] ? a.gamma[c0 + i] : 1.0f;
      ag[j][i] = ab[j][i] = 0.0f;
    }
  }
  const float inv_d = 1.0f / float(d);
  for (int64_t r0 = int64_t(blockIdx.x) * kRows; r0 < a.rows; r0 += int64_t(gridDim.x) * kRows) {
    const int64_t r = r0 + threadIdx.x / L;
    const bool live = r < a.rows;
    const float mean = live ? a.mean[r] : 0.0f, rstd = live ? a.rstd[r] : 0.0f;
    float xh[C][K], g[C][K];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int64_t at = (l + L * j) * K;
      const Chunk<T> cx = load_chunk_n(x + r * a.ldx + at, live ? n[j] : 0);
      const Chunk<T> cy = load_chunk_n(dy + r * a.lddy + at, live ? n[j] : 0);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float u = float(cy.v[i]);
        xh[j][i] = live && i < n[j] ? (float(cx.v[i]) - mean) * rstd : 0.0f;
        ag[j][i] = fmaf(u, xh[j][i], ag[j][i]);
        ab[j][i] += u;
        g[j][i] = u * gm[j][i];
        s1 += g[j][i];
        s2 = fmaf(g[j][i], xh[j][i], s2);
      }
    }
    if (dx == nullptr) continue;
    s1 = row_sum<L>(s1, s) * inv_d;
    s2 = row_sum<L>(s2, s) * inv_d;
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (n[j] == 0) continue;
      const int64_t at = (l + L * j) * K;
      Chunk<T> cr, c;
      if (dres != nullptr) cr = load_chunk_n(dres + r * a.lddres + at, n[j]);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float o = rstd * (g[j][i] - s1 - xh[j][i] * s2);
        if (dres != nullptr) o += float(cr.v[i]);
        c.v[i] = T(o);
      }
      store_chunk_n(dx + r * a.lddx + at, c, n[j]);
    }
  }
  if (part == nullptr) return;
  float* __restrict__ out = part + size_t(blockIdx.x) * 2 * d;
  // the workgroup's rows, in a fixed order: lanes of a wave, then the waves
  constexpr int LW = L < 64 ? L : 64;
  __shared__ float sw[L > 64 ? 1 : 4][LW * K];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float v[K];
#pragma unroll
      for (int i = 0; i < K; ++i) {
        v[i] = which == 0 ? ag[j][i] : ab[j][i];
#pragma unroll
        for (int o = LW; o < 64; o <<= 1) v[i] += __shfl_xor(v[i], o, 64);
      }
      if constexpr (L > 64) {
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (i < n[j]) out[which * d + (l + L * j) * K + i] = v[i];
      } else {
        __syncthreads();
        if ((threadIdx.x & 63) < LW)
#pragma unroll
          for (int i = 0; i < K; ++i) sw[threadIdx.x >> 6][l * K + i] = v[i];
        __syncthreads();
        for (int i = threadIdx.x; i < LW * K; i += kThreads) {
          const int col = L * j * K + i;
          if (col < d) out[which * d + col] = (sw[0][i] + sw[1][i]) + (sw[2][i] + sw[3][i]);
        }
      }
    }
}

// Rows wider than the registers of a workgroup: the row is read again (from
// L2) for each sum.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_fwd_wide(NormArgs a) {
  constexpr int K = kChunk<T>;
  __shared__ float s[4];
  const float inv_d = 1.0f / float(a.width);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* __restrict__ x = static_cast<const T*>(a.x) + r * a.ldx;
    T* __restrict__ y = static_cast<T*>(a.y) + r * a.ldy;
    float sum = 0.0f, sq = 0.0f;
    for (int c = threadIdx.x * K; c < a.width; c += kThreads * K) {
      const Chunk<T> v = load_chunk_n(x + c, a.width - c);
#pragma unroll
      for (int i = 0; i < K; ++i) sum += float(v.v[i]);
    }
    const float mean = row_sum<256>(sum, s) * inv_d;
    for (int c = threadIdx.x * K; c < a.width; c += kThreads * K) {
      const Chunk<T> v = load_chunk_n(x + c, a.width - c);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float u = c + i < a.width ? float(v.v[i]) - mean : 0.0f;
        sq = fmaf(u, u, sq);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<256>(sq, s) * inv_d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[r] = mean;
      if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
    for (int c = threadIdx.x * K; c < a.width; c += kThreads * K) {
      const Chunk<T> v = load_chunk_n(x + c, a.width - c);
      Chunk<T> o;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const bool in = c + i < a.width;
        const float gm = in && a.gamma != nullptr ? a.gamma[c + i] : 1.0f;
        const float bt = in && a.beta != nullptr ? a.beta[c + i] : 0.0f;
        o.v[i] = T(fmaf((float(v.v[i]) - mean) * rstd, gm, bt));
      }
      store_chunk_n(y + c, o, a.width - c);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_dx_wide(NormArgs a) {
  constexpr int K = kChunk<T>;
  __shared__ float s[4];
  const float inv_d = 1.0f / float(a.width);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* __restrict__ x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* __restrict__ dy = static_cast<const T*>(a.dy) + r * a.lddy;
    T* __restrict__ dx = static_cast<T*>(a.dx) + r * a.lddx;
    const T* __restrict__ dres = a.dres != nullptr ? static_cast<const T*>(a.dres) + r * a.lddres : nullptr;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x * K; c < a.width; c += kThreads * K) {
      const Chunk<T> cx = load_chunk_n(x + c, a.width - c), cy = load_chunk_n(dy + c, a.width - c);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const bool in = c + i < a.width;
        const float g = float(cy.v[i]) * (in && a.gamma != nullptr ? a.gamma[c + i] : 1.0f);
        s1 += g;
        s2 = fmaf(g, in ? (float(cx.v[i]) - mean) * rstd : 0.0f, s2);
      }
    }
    s1 = row_sum<256>(s1, s) * inv_d;
    s2 = row_sum<256>(s2, s) * inv_d;
    for (int c = threadIdx.x * K; c < a.width; c += kThreads * K) {
      const Chunk<T> cx = load_chunk_n(x + c, a.width - c), cy = load_chunk_n(dy + c, a.width - c);
      Chunk<T> cr, o;
      if (dres != nullptr) cr = load_chunk_n(dres + c, a.width - c);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const bool in = c + i < a.width;
        const float g = float(cy.v[i]) * (in && a.gamma != nullptr ? a.gamma[c + i] : 1.0f);
        float v = rstd * (g - s1 - (float(cx.v[i]) - mean) * rstd * s2);
        if (dres != nullptr) v += float(cr.v[i]);
        o.v[i] = T(v);
      }
      store_chunk_n(dx + c, o, a.width - c);
    }
  }
}

// Column sums of the wide case: workgroup (column stretch, row share).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_cols_wide(NormArgs a, float* __restrict__ part) {
  constexpr int K = kChunk<T>;
  const int c = (blockIdx.x * kThreads + threadIdx.x) * K;
  if (c >= a.width) return;
  const int64_t share = (int64_t(a.rows) + gridDim.y - 1) / gridDim.y;
  const int64_t r0 = blockIdx.y * share, r1 = std::min<int64_t>(a.rows, r0 + share);
  float ag[K], ab[K];
#pragma unroll
  for (int i = 0; i < K; ++i) ag[i] = ab[i] = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const Chunk<T> cx = load_chunk_n(static_cast<const T*>(a.x) + r * a.ldx + c, a.width - c);
    const Chunk<T> cy = load_chunk_n(static_cast<const T*>(a.dy) + r * a.lddy + c, a.width - c);
    const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float u = float(cy.v[i]);
      ag[i] = fmaf(u, (float(cx.v[i]) - mean) * rstd, ag[i]);
      ab[i] += u;
    }
  }
  float* __restrict__ out = part + size_t(blockIdx.y) * 2 * a.width;
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (c + i < a.width) {
      out[c + i] = ag[i];
      out[a.width + c + i] = ab[i];
    }
}

// Sums the partial rows: 64 columns a workgroup, 16 shares of the partial
// rows, joined in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_reduce(const float* __restrict__ part, int parts, int width,
                                                      float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float s[16][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
  float v = 0.0f;
  if (col < 2 * width)
#pragma unroll 8
    for (int p = w; p < parts; p += 16) v += part[size_t(p) * 2 * width + col];
  s[w][threadIdx.x & 63] = v;
  __syncthreads();
  if (w != 0 || col >= 2 * width) return;
  v = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += s[k][threadIdx.x];
  if (col < width) {
    if (dgamma != nullptr) dgamma[col] = v;
  } else if (dbeta != nullptr) {
    dbeta[col - width] = v;
  }
}

int wide_shares(int64_t rows, int32_t width) {
  const int64_t cols = (int64_t(width) + 1023) / 1024;   // workgroups across, fp32 chunks
  return int(std::min<int64_t>(std::max<int64_t>(rows, 1), std::max<int64_t>(1, kBwdGroups / cols)));
}

template <typename T, int L, int C>
hipError_t go_fwd(const NormArgs& a, hipStream_t st) {
  const int64_t blocks = (int64_t(a.rows) + kThreads / L - 1) / (kThreads / L);
  k_norm_fwd<T, L, C><<<int(std::min<int64_t>(blocks, kFwdGroups)), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int L, int C>
hipError_t go_bwd(const NormArgs& a, float* part, hipStream_t st) {
  const int64_t blocks = (int64_t(a.rows) + kThreads / L - 1) / (kThreads / L);
  const int grid = int(std::max<int64_t>(1, std::min<int64_t>(blocks, kBwdGroups)));
  const bool sums = a.dgamma != nullptr || a.dbeta != nullptr;
  k_norm_bwd<T, L, C><<<grid, kThreads, 0, st>>>(a, sums ? part : nullptr);
  if (sums)
    k_norm_reduce<<<(2 * a.width + 63) / 64, 1024, 0, st>>>(part, grid, a.width, a.dgamma, a.dbeta);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_fwd(const NormArgs& a, hipStream_t st) {
  const int chunks = (a.width + kChunk<T> - 1) / kChunk<T>;
  if (chunks <= 8) return go_fwd<T, 8, 1>(a, st);
  if (chunks <= 16) return go_fwd<T, 16, 1>(a, st);
  if (chunks <= 32) return go_fwd<T, 32, 1>(a, st);
  if (chunks <= 64) return go_fwd<T, 64, 1>(a, st);
  if (chunks <= 128) return go_fwd<T, 64, 2>(a, st);
  if (chunks <= 192) return go_fwd<T, 64, 3>(a, st);
  if (chunks <= 256) return go_fwd<T, 64, 4>(a, st);
  if (chunks <= 512) return go_fwd<T, 256, 2>(a, st);
  if (chunks <= 1024) return go_fwd<T, 256, 4>(a, st);
  k_norm_fwd_wide<T><<<int(std::min<int64_t>(a.rows, kFwdGroups)), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd(const NormArgs& a, float* part, hipStream_t st) {
  const int chunks = (a.width + kChunk<T> - 1) / kChunk<T>;
  if (chunks <= 8) return go_bwd<T, 8, 1>(a, part, st);
  if (chunks <= 16) return go_bwd<T, 16, 1>(a, part, st);
  if (chunks <= 32) return go_bwd<T, 32, 1>(a, part, st);
  if (chunks <= 64) return go_bwd<T, 64, 1>(a, part, st);
  if (chunks <= 128) return go_bwd<T, 64, 2>(a, part, st);
  if (chunks <= 192) return go_bwd<T, 64, 3>(a, part, st);
  if (chunks <= 256) return go_bwd<T, 64, 4>(a, part, st);
  if (chunks <= 512) return go_bwd<T, 256, 2>(a, part, st);
  if (chunks <= 1024) return go_bwd<T, 256, 4>(a, part, st);
  if (a.rows > 0 && a.dx != nullptr)
    k_norm_dx_wide<T><<<int(std::min<int64_t>(a.rows, kFwdGroups)), kThreads, 0, st>>>(a);
  if (a.dgamma != nullptr || a.dbeta != nullptr) {
    const int shares = wide_shares(a.rows, a.width);
    const int across = (a.width + kThreads * kChunk<T> - 1) / (kThreads * kChunk<T>);
    k_norm_cols_wide<T><<<dim3(across, shares), kThreads, 0, st>>>(a, part);
    k_norm_reduce<<<(2 * a.width + 63) / 64, 1024, 0, st>>>(part, shares, a.width, a.dgamma, a.dbeta);
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace net

size_t layer_norm_ws_bytes(int64_t rows, int32_t width) {
  // partial rows: at most kBwdGroups, and no more than there are rows
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(rows, net::kBwdGroups));
  return align_up(size_t(parts) * 2 * size_t(width) * sizeof(float), 256);
}

hipError_t launch_layer_norm_fwd(int type, const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (type == kTypeBF16) return net::norm_fwd<net::bf16>(a, st);
  if (type == kTypeF16) return net::norm_fwd<net::f16>(a, st);
  return net::norm_fwd<float>(a, st);
}

hipError_t launch_layer_norm_bwd(int type, const NormArgs& a, void* ws, hipStream_t st) {
  float* part = static_cast<float*>(ws);
  if (type == kTypeBF16) return net::norm_bwd<net::bf16>(a, part, st);
  if (type == kTypeF16) return net::norm_bwd<net::f16>(a, part, st);
  return net::norm_bwd<float>(a, part, st);
}

}  // namespace gs
