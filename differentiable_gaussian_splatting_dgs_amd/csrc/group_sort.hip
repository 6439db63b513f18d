// Stable sort of group ids, with the groups' bounds: what rows routed to
// heads, and the gradient of a shared feature table, are laid out by.
//
// An id becomes a key in [0, G], G for an id of no group.  Keys are sorted by
// digits of up to kMaxBits bits, least significant first, each pass stable:
// digit counts of every block of keys, a scan of each digit's counts over the
// blocks, then the keys to their places, ranked within the block by wave
// ballots.  Up to 1023 groups that is one pass, whose digits are the groups
// and whose counts are the bounds; more groups take the bounds from the sorted
// keys by bisection.  No workgroup waits on another, nothing is counted by
// global atomics: the same ids give the same order.
//
// Bound by latency below some 100,000 ids (the launches), by the scattered
// writes of order and place above.
#include <algorithm>
#include <type_traits>

#include "gs_scan.hpp"

namespace gs {
namespace {

constexpr int kT = 256;              // threads of a block
constexpr int kW = kT / 64;
constexpr int kItems = 8;            // keys of a thread
constexpr int kBlockKeys = kT * kItems;
constexpr int kMaxBits = 10;         // of a digit

template <typename I>
__device__ __forceinline__ uint32_t key_of(I id, uint32_t groups) {
  // as an unsigned number a negative id is past every group too
  using U = std::make_unsigned_t<I>;
  return U(id) < U(groups) ? uint32_t(id) : groups;
}

// The first pass reads ids, the later ones keys.
template <typename I, bool kFirst>
__device__ __forceinline__ uint32_t load_key(const void* __restrict__ src, int64_t i, uint32_t groups) {
  if constexpr (kFirst)
    return key_of(static_cast<const I*>(src)[i], groups);
  else
    return static_cast<const uint32_t*>(src)[i];
}

// counts[digit][block]
template <typename I, bool kFirst, int kBits>
__global__ __launch_bounds__(kT) void k_count(const void* __restrict__ src, int64_t n, uint32_t groups, int shift,
                                              uint32_t* __restrict__ counts, int nb) {
  constexpr int kBins = 1 << kBits;
  __shared__ uint32_t hist[kBins];
  for (int b = threadIdx.x; b < kBins; b += kT) hist[b] = 0;
  __syncthreads();
  const int64_t base = int64_t(blockIdx.x) * kBlockKeys + threadIdx.x;
  uint32_t d[kItems];
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int64_t i = base + it * kT;
    d[it] = i < n ? (load_key<I, kFirst>(src, i, groups) >> shift) & (kBins - 1) : 0u;
  }
#pragma unroll
  for (int it = 0; it < kItems; ++it)
    if (base + it * kT < n) atomicAdd(&hist[d[it]], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += kT) counts[size_t(b) * nb + blockIdx.x] = hist[b];
}

// One workgroup for each digit: its counts become the keys of that digit in
// the blocks before, its total goes to totals.
__global__ __launch_bounds__(kT) void k_scan(uint32_t* __restrict__ counts, int nb, uint32_t* __restrict__ totals) {
  __shared__ uint32_t sh[kW];
  uint32_t* row = counts + size_t(blockIdx.x) * nb;
  uint32_t carry = 0;
  for (int base = 0; base < nb; base += kT) {
    const int i = base + int(threadIdx.x);
    const uint32_t v = i < nb ? row[i] : 0u;
    uint32_t tot;
    const uint32_t ex = block_exclusive_scan<kT, uint32_t>(v, sh, tot);
    if (i < nb) row[i] = carry + ex;
    carry += tot;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

struct Pass {
  const void* keys;              // ids in the first pass
  const uint32_t* entries;       // NULL in the first pass: 0, 1, ...
  uint32_t* out_keys;            // NULL if nothing reads them
  uint32_t* out_entries;         // order in the last pass, or NULL
  int32_t* place;                // last pass, or NULL
  int64_t* offsets;              // the only pass: written here; else NULL
  const uint32_t* counts;
  const uint32_t* totals;
  int64_t n;
  uint32_t groups;
  int32_t shift, nb;
};

// Each key of the block to its place: the keys of smaller digits, those of
// its digit in the blocks before, and those before it in the block.
template <typename I, bool kFirst, int kBits>
__global__ __launch_bounds__(kT) void k_place(Pass p) {
  constexpr int kBins = 1 << kBits;
  __shared__ uint32_t s_cnt[kW][kBins];     // per-wave running counts, then the wave's first place
  __shared__ uint32_t s_scan[kW];
  const int t = threadIdx.x, w = t >> 6, lane = t & 63;
  const int64_t base = int64_t(blockIdx.x) * kBlockKeys + w * (kItems * 64) + lane;
  uint32_t key[kItems], rank[kItems], entry[kItems];
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int64_t i = base + it * 64;
    key[it] = i < p.n ? load_key<I, kFirst>(p.keys, i, p.groups) : 0u;
    entry[it] = kFirst ? uint32_t(i) : (i < p.n ? p.entries[i] : 0u);
  }
  for (int b = t; b < kW * kBins; b += kT) (&s_cnt[0][0])[b] = 0;
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const bool valid = base + it * 64 < p.n;
    const uint32_t d = (key[it] >> p.shift) & (kBins - 1);
    const uint64_t peers = match_bits<kBits>(d, ballot(valid));
    const uint32_t below = uint32_t(count_below(peers));
    const uint32_t prior = s_cnt[w][d];
    rank[it] = prior + below;
    __builtin_amdgcn_wave_barrier();
    if (valid && below == 0) s_cnt[w][d] = prior + uint32_t(__popcll(peers));
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // thread t: kPer neighbouring digits
  constexpr int kPer = (kBins + kT - 1) / kT;
  uint32_t tot[kPer], mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = t * kPer + j;
    tot[j] = b < kBins ? p.totals[b] : 0u;
    mine += tot[j];
  }
  uint32_t all;
  uint32_t start = block_exclusive_scan<kT, uint32_t>(mine, s_scan, all);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = t * kPer + j;
    if (b < kBins) {
      if (p.offsets != nullptr && blockIdx.x == 0 && uint32_t(b) <= p.groups) p.offsets[b] = start;
      uint32_t at = start + p.counts[size_t(b) * p.nb + blockIdx.x];
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const uint32_t c = s_cnt[k][b];
        s_cnt[k][b] = at;
        at += c;
      }
      start += tot[j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    if (base + it * 64 >= p.n) continue;
    const uint32_t d = (key[it] >> p.shift) & (kBins - 1);
    const uint32_t at = s_cnt[w][d] + rank[it];
    if (p.out_keys != nullptr) p.out_keys[at] = key[it];
    if (p.out_entries != nullptr) p.out_entries[at] = entry[it];
    if (p.place != nullptr) p.place[entry[it]] = key[it] < p.groups ? int32_t(at) : -1;
  }
}

// offsets[g] = the first position whose key is at least g.
__global__ __launch_bounds__(kT) void k_bounds(const uint32_t* __restrict__ keys, int64_t n, int64_t groups,
                                               int64_t* __restrict__ offsets) {
  const int64_t g = int64_t(blockIdx.x) * kT + threadIdx.x;
  if (g > groups) return;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (int64_t(keys[mid]) < g)
      lo = mid + 1;
    else
      hi = mid;
  }
  offsets[g] = lo;
}

int key_bits(int64_t groups) {      // of a key in [0, groups]
  int b = 1;
  while ((groups >> b) != 0) ++b;
  return b;
}

struct SortSpace {
  uint32_t *counts, *totals, *keys[2], *entries[2];
  size_t bytes;
};

SortSpace sort_space(void* ws, int64_t n, int64_t groups) {
  const int64_t nb = (n + kBlockKeys - 1) / kBlockKeys;
  const bool many = key_bits(groups) > kMaxBits;
  char* p = static_cast<char*>(ws);
  SortSpace s{};
  auto take = [&](size_t words) {
    uint32_t* at = reinterpret_cast<uint32_t*>(p + s.bytes);
    s.bytes += align_up(words * 4, 256);
    return at;
  };
  s.counts = take(size_t(nb) << kMaxBits);
  s.totals = take(size_t(1) << kMaxBits);
  if (many)
    for (int k = 0; k < 2; ++k) {
      s.keys[k] = take(size_t(n));
      s.entries[k] = take(size_t(n));
    }
  return s;
}

template <typename I, bool kFirst, int kBits>
void pass(const Pass& p, const SortSpace& s, hipStream_t st) {
  k_count<I, kFirst, kBits><<<p.nb, kT, 0, st>>>(p.keys, p.n, p.groups, p.shift, s.counts, p.nb);
  k_scan<<<1 << kBits, kT, 0, st>>>(s.counts, p.nb, s.totals);
  k_place<I, kFirst, kBits><<<p.nb, kT, 0, st>>>(p);
}

template <typename I>
hipError_t sort(const SortArgs& a, void* ws, hipStream_t st) {
  if (a.n == 0) {
    k_bounds<<<unsigned((a.groups + kT) / kT), kT, 0, st>>>(nullptr, 0, a.groups, a.offsets);
    return hipGetLastError();
  }
  const SortSpace s = sort_space(ws, a.n, a.groups);
  const int bits = key_bits(a.groups);
  const int passes = (bits + kMaxBits - 1) / kMaxBits;
  const int digit = std::max(8, (bits + passes - 1) / passes);
  Pass p{};
  p.keys = a.ids;
  p.n = a.n;
  p.groups = uint32_t(a.groups);
  p.nb = int((a.n + kBlockKeys - 1) / kBlockKeys);
  p.counts = s.counts;
  p.totals = s.totals;
  for (int k = 0; k < passes; ++k) {
    const bool last = k == passes - 1;
    p.shift = k * digit;
    p.out_keys = passes > 1 ? s.keys[k & 1] : nullptr;
    p.out_entries = last ? reinterpret_cast<uint32_t*>(a.order) : s.entries[k & 1];
    p.place = last ? a.place : nullptr;
    p.offsets = passes == 1 ? a.offsets : nullptr;
    if (k == 0) {
      digit == 8 ? pass<I, true, 8>(p, s, st) : digit == 9 ? pass<I, true, 9>(p, s, st) : pass<I, true, 10>(p, s, st);
    } else {
      digit == 8 ? pass<I, false, 8>(p, s, st)
                 : digit == 9 ? pass<I, false, 9>(p, s, st) : pass<I, false, 10>(p, s, st);
    }
    p.keys = p.out_keys;
    p.entries = p.out_entries;
  }
  if (passes > 1)
    k_bounds<<<unsigned((a.groups + kT) / kT), kT, 0, st>>>(static_cast<const uint32_t*>(p.keys), a.n, a.groups,
                                                            a.offsets);
  return hipGetLastError();
}

}  // namespace

size_t group_sort_ws_bytes(int64_t n, int64_t groups) { return sort_space(nullptr, n, groups).bytes; }

hipError_t launch_group_sort(const SortArgs& a, void* ws, hipStream_t st) {
  return a.id_bytes == 4 ? sort<int32_t>(a, ws, st) : sort<int64_t>(a, ws, st);
}

}  // namespace gs
