// Stable sort of group ids, with the groups' bounds: what rows routed to
// heads, and the gradient of a shared feature table, are laid out by.
//
// An id becomes a key in [0, G], G for an id of no group.  Keys are sorted by
// digits, least significant first, each pass stable; within a block a key's
// rank among the keys of its digit comes from wave ballots.
//
// Up to kSmall keys: one workgroup, all passes in LDS, one launch (and one for
// the bounds of many groups), so that a few hundred routed rows cost a launch.
// More keys: a pass is three launches, the digit counts of every block of
// keys, a scan of each digit's counts over the blocks (left out for few
// blocks), and the keys to their places.  A block's keys are brought into the digits' order in LDS first and
// leave as runs of one digit, key and entry as one 8-byte word, instead of
// one by one.  Up to 1023 groups that is one pass, whose digits are the
// groups and whose counts are the bounds; more groups take the bounds from
// the sorted keys by bisection.  No workgroup waits on another, nothing is
// counted by global atomics: the same ids give the same order.
//
// Bound by latency, of launches and of the phases within one: 1,000,000 ids of
// 100,000 groups take 54 us in seven launches (counts 7 + 6, scans 5 + 4, places 11
// + 11, bounds 8 to 9 us; the bytes alone 13), 800,000 ids of 16 groups 20 us in
// three, 8,191 ids of 50,021 groups 17 + 4 us, 6 ids of 64 groups 2.7 us.  Blocks of
// 2048 keys (of 256 threads) instead of 4096: 8 us more in all, of 8192 4 us.
#include <algorithm>
#include <type_traits>

#include "gs_scan.hpp"

namespace gs {
namespace {

template <typename I>
__device__ __forceinline__ uint32_t key_of(I id, uint32_t groups) {
  // as an unsigned number a negative id is past every group too
  using U = std::make_unsigned_t<I>;
  return U(id) < U(groups) ? uint32_t(id) : groups;
}

// The lanes among `act` with this lane's digit of `bits` bits (bits is the
// same for the whole wave).
__device__ __forceinline__ uint64_t match_digit(uint32_t d, int bits, uint64_t act) {
  uint32_t lo = uint32_t(act), hi = uint32_t(act >> 32);
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    if (b >= bits) break;
    const int32_t mine = int32_t(d << (31 - b)) >> 31;      // the bit in all places
    const uint64_t set = ballot(mine != 0);
    lo &= ~(uint32_t(set) ^ uint32_t(mine));
    hi &= ~(uint32_t(set >> 32) ^ uint32_t(mine));
  }
  return uint64_t(hi) << 32 | lo;
}

// --- one workgroup --------------------------------------------------------------------

constexpr int kSmall = 8192;
constexpr int kSmallBits = 8;
constexpr int kSmallBounds = 8192;      // groups whose bounds the workgroup writes itself

template <typename I, int NT, int NI>
__global__ __launch_bounds__(NT) void k_sort_small(SortArgs a, int bits, int passes, uint32_t* __restrict__ sorted) {
  constexpr int kW = NT / 64, kBins = 1 << kSmallBits;
  __shared__ uint32_t s_key[NT * NI];
  __shared__ uint16_t s_entry[NT * NI];
  __shared__ uint32_t s_cnt[kW][kBins];
  __shared__ uint32_t s_scan[kW];
  const int t = threadIdx.x, w = t >> 6, lane = t & 63;
  const int n = int(a.n), first = w * (NI * 64) + lane;
  const uint32_t groups = uint32_t(a.groups);
  const int digit = (bits + passes - 1) / passes, bins = 1 << digit;
  uint32_t key[NI], entry[NI], rank[NI];
#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = first + it * 64;
    key[it] = i < n ? key_of(static_cast<const I*>(a.ids)[i], groups) : 0u;
    entry[it] = uint32_t(i);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * digit;
    for (int b = lane; b < bins; b += 64) s_cnt[w][b] = 0;
    __builtin_amdgcn_wave_barrier();      // a wave's counts are its own
#pragma unroll
    for (int it = 0; it < NI; ++it) {
      const bool valid = first + it * 64 < n;
      const uint32_t d = (key[it] >> shift) & uint32_t(bins - 1);
      const uint64_t peers = match_digit(d, digit, ballot(valid));
      const uint32_t below = uint32_t(count_below(peers));
      const uint32_t prior = s_cnt[w][d];
      rank[it] = prior + below;
      __builtin_amdgcn_wave_barrier();
      if (valid && below == 0) s_cnt[w][d] = prior + uint32_t(__popcll(peers));
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // counts to first places: digit t of every wave (bins <= NT)
    uint32_t c[kW], mine = 0;
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      c[k] = t < bins ? s_cnt[k][t] : 0u;
      mine += c[k];
    }
    uint32_t all;
    uint32_t at = block_exclusive_scan<NT, uint32_t>(mine, s_scan, all);
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      if (t < bins) s_cnt[k][t] = at;
      at += c[k];
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < NI; ++it)
      if (first + it * 64 < n) {
        const uint32_t d = (key[it] >> shift) & uint32_t(bins - 1);
        const uint32_t p = s_cnt[w][d] + rank[it];
        s_key[p] = key[it];
        s_entry[p] = uint16_t(entry[it]);
      }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < NI; ++it) {
      const int i = first + it * 64;
      if (i < n) {
        key[it] = s_key[i];
        entry[it] = s_entry[i];
      }
    }
  }
#pragma unroll
  for (int it = 0; it < NI; ++it) {
    const int i = first + it * 64;
    if (i >= n) continue;
    if (a.order != nullptr) a.order[i] = int32_t(entry[it]);
    if (a.place != nullptr) a.place[entry[it]] = key[it] < groups ? i : -1;
    if (sorted != nullptr) sorted[i] = key[it];
  }
  if (sorted != nullptr) return;
  // the first place whose key is at least g (the last pass ends with the keys
  // in LDS, behind a barrier)
  for (uint32_t g = t; g <= groups; g += NT) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_key[mid] < g)
        lo = mid + 1;
      else
        hi = mid;
    }
    a.offsets[g] = lo;
  }
}

// --- many blocks ------------------------------------------------------------------------

constexpr int kT = 512;              // threads of a block
constexpr int kW = kT / 64;
constexpr int kItems = 8;            // keys of a thread
constexpr int kBlockKeys = kT * kItems;
constexpr int kMaxBits = 10;         // of a digit
constexpr int kFewBlocks = 32;       // so many blocks' counts are read by each instead of scanned by a launch

struct Pass {
  const void* src;               // ids in the first pass, then keys and entries as words
  uint64_t* out;                 // words of the next pass; NULL in the last one
  uint32_t* out_keys;            // last of several passes: sorted keys; else NULL
  int32_t* order;                // last pass, or NULL
  int32_t* place;                // last pass, or NULL
  int64_t* offsets;              // the only pass: written here; else NULL
  uint32_t* counts;              // [block][digit]
  uint32_t* totals;              // NULL: few blocks, whose counts are not scanned
  int64_t n;
  uint32_t groups;
  int32_t shift, bits, nb;
};

// The first pass reads ids, the later ones words of entry and key.
template <typename I, bool kFirst>
__device__ __forceinline__ uint64_t load_word(const void* __restrict__ src, int64_t i, uint32_t groups) {
  if constexpr (kFirst)
    return uint64_t(i) << 32 | key_of(static_cast<const I*>(src)[i], groups);
  else
    return static_cast<const uint64_t*>(src)[i];
}

template <typename I, bool kFirst>
__global__ __launch_bounds__(kT) void k_count(Pass p) {
  __shared__ uint32_t hist[1 << kMaxBits];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kT) hist[b] = 0;
  __syncthreads();
  const int64_t base = int64_t(blockIdx.x) * kBlockKeys + threadIdx.x;
  uint32_t d[kItems];
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int64_t i = base + it * kT;
    d[it] = i < p.n ? (uint32_t(load_word<I, kFirst>(p.src, i, p.groups)) >> p.shift) & uint32_t(bins - 1) : 0u;
  }
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const bool valid = base + it * kT < p.n;
    if (p.bits <= 6) {      // few digits: most lanes would add to the same ones
      const uint64_t peers = match_digit(d[it], p.bits, ballot(valid));
      if (valid && count_below(peers) == 0) atomicAdd(&hist[d[it]], uint32_t(__popcll(peers)));
    } else if (valid) {
      atomicAdd(&hist[d[it]], 1u);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kT) p.counts[(size_t(blockIdx.x) << p.bits) + b] = hist[b];
}

// 64 digits a workgroup, a lane each: a digit's counts become its keys in the
// blocks before, its total goes to totals.  Every wave takes a stretch of the
// blocks, sums it, and counts on from the stretches before.
__global__ __launch_bounds__(1024) void k_scan(uint32_t* __restrict__ counts, int bits, int nb,
                                               uint32_t* __restrict__ totals) {
  __shared__ uint32_t sh[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, d = blockIdx.x * 64 + lane;
  const bool live = d < (1 << bits);
  constexpr int kHeld = 16;
  const int each = (nb + 15) / 16, b0 = std::min(w * each, nb), b1 = std::min(b0 + each, nb);
  uint32_t sum = 0, held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    held[i] = live && b0 + i < b1 ? counts[(size_t(b0 + i) << bits) + d] : 0u;
    sum += held[i];
  }
  if (live)
#pragma unroll 8
    for (int b = b0 + kHeld; b < b1; ++b) sum += counts[(size_t(b) << bits) + d];
  sh[w][lane] = sum;
  __syncthreads();
  uint32_t at = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t c = sh[k][lane];
    at += k < w ? c : 0u;
    all += c;
  }
  if (!live) return;
  if (w == 0) totals[d] = all;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (b0 + i < b1) counts[(size_t(b0 + i) << bits) + d] = at;
    at += held[i];
  }
#pragma unroll 8
  for (int b = b0 + kHeld; b < b1; ++b) {
    uint32_t* const c = counts + (size_t(b) << bits) + d;
    const uint32_t mine = *c;
    *c = at;
    at += mine;
  }
}

// Each key of the block to its place: behind the keys of smaller digits, those
// of its digit in the blocks before, and those before it in the block.
template <typename I, bool kFirst>
__global__ __launch_bounds__(kT) void k_place(Pass p) {
  constexpr int kMaxBins = 1 << kMaxBits, kPer = kMaxBins / kT;
  __shared__ uint64_t s_word[kBlockKeys];
  __shared__ uint16_t s_cnt[kW][kMaxBins];      // a wave's counts, then its first places in the block
  __shared__ uint32_t s_to[kMaxBins];           // a digit's first place, less its first one in the block
  __shared__ uint32_t s_scan[kW];
  const int t = threadIdx.x, w = t >> 6, lane = t & 63, bins = 1 << p.bits;
  const int64_t block = int64_t(blockIdx.x) * kBlockKeys;
  const int n = int(std::min<int64_t>(kBlockKeys, p.n - block)), first = w * (kItems * 64) + lane;
  uint64_t word[kItems];
  uint32_t rank[kItems];
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int i = first + it * 64;
    word[it] = i < n ? load_word<I, kFirst>(p.src, block + i, p.groups) : 0u;
  }
  // thread t: what it has to know of kPer neighbouring digits, on its way while
  // the keys are ranked
  uint32_t tot[kPer], before[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = t * kPer + j;
    tot[j] = before[j] = 0;
    if (b < bins && p.totals != nullptr) {
      tot[j] = p.totals[b];
      before[j] = p.counts[(size_t(blockIdx.x) << p.bits) + b];
    } else if (b < bins) {
#pragma unroll 8
      for (int k = 0; k < p.nb; ++k) {
        const uint32_t c = p.counts[(size_t(k) << p.bits) + b];
        tot[j] += c;
        before[j] += k < int(blockIdx.x) ? c : 0u;
      }
    }
  }
  for (int b = lane; b < bins; b += 64) s_cnt[w][b] = 0;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const bool valid = first + it * 64 < n;
    const uint32_t d = (uint32_t(word[it]) >> p.shift) & uint32_t(bins - 1);
    const uint64_t peers = match_digit(d, p.bits, ballot(valid));
    const uint32_t below = uint32_t(count_below(peers));
    const uint32_t prior = s_cnt[w][d];
    rank[it] = prior + below;
    __builtin_amdgcn_wave_barrier();
    if (valid && below == 0) s_cnt[w][d] = uint16_t(prior + uint32_t(__popcll(peers)));
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // thread t: kPer neighbouring digits
  uint32_t in_block[kPer], tot_sum = 0, block_sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = t * kPer + j;
    in_block[j] = 0;
    if (b < bins)
#pragma unroll
      for (int k = 0; k < kW; ++k) in_block[j] += s_cnt[k][b];
    tot_sum += tot[j];
    block_sum += in_block[j];
  }
  uint32_t all;
  uint32_t start = block_exclusive_scan<kT, uint32_t>(tot_sum, s_scan, all);
  uint32_t local = block_exclusive_scan<kT, uint32_t>(block_sum, s_scan, all);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = t * kPer + j;
    if (b < bins) {
      if (p.offsets != nullptr && blockIdx.x == 0 && uint32_t(b) <= p.groups) p.offsets[b] = start;
      s_to[b] = start + before[j] - local;
      uint32_t at = local;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const uint32_t c = s_cnt[k][b];
        s_cnt[k][b] = uint16_t(at);
        at += c;
      }
      start += tot[j];
      local += in_block[j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kItems; ++it)
    if (first + it * 64 < n) {
      const uint32_t key = uint32_t(word[it]), d = (key >> p.shift) & uint32_t(bins - 1);
      const uint32_t at = s_cnt[w][d] + rank[it];
      s_word[at] = word[it];
      // entries of the first pass are neighbours, as their places are then
      if (kFirst && p.place != nullptr)
        p.place[word[it] >> 32] = key < p.groups ? int32_t(s_to[d] + at) : -1;
    }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kItems; ++it) {
    const int i = it * kT + t;
    if (i >= n) continue;
    const uint64_t v = s_word[i];
    const uint32_t key = uint32_t(v), at = s_to[(key >> p.shift) & uint32_t(bins - 1)] + uint32_t(i);
    if (p.out != nullptr) p.out[at] = v;
    if (p.out_keys != nullptr) p.out_keys[at] = key;
    if (p.order != nullptr) p.order[at] = int32_t(v >> 32);
    if (!kFirst && p.place != nullptr) p.place[v >> 32] = key < p.groups ? int32_t(at) : -1;
  }
}

// offsets[g] = the first position whose key is at least g.  A workgroup's
// bounds lie between those of its first and its last group, which its first and
// its last two waves find with 128 keys a step.  Each thread goes on in LDS, or, where an id
// of very many entries is among them, in memory with 3 keys a step.
__global__ __launch_bounds__(256) void k_bounds(const uint32_t* __restrict__ keys, int64_t n, int64_t groups,
                                                int64_t* __restrict__ offsets) {
  constexpr int kHeld = 4096;
  __shared__ int s_smaller[2][4];
  __shared__ int64_t s_ends[2];
  __shared__ uint32_t s_key[kHeld];
  const int64_t g0 = int64_t(blockIdx.x) * 256, g = g0 + threadIdx.x;
  {
    // keys before lo are smaller, keys from hi on are not
    const int w = threadIdx.x >> 6, i = threadIdx.x & 127;
    const int64_t want = g0 + (w >> 1) * 256;
    int64_t lo = 0, hi = n;
    for (int64_t left = n, turn = 0; left > 0; left = (left + 127) / 128 - 1, ++turn) {      // as long for both
      const int64_t step = (hi - lo + 127) / 128, at = lo + i * step;
      const uint64_t smaller = ballot(lo < hi && at < hi && int64_t(keys[at < hi ? at : lo]) < want);
      if ((threadIdx.x & 63) == 0) s_smaller[turn & 1][w] = __popcll(smaller);
      __syncthreads();
      const int k = s_smaller[turn & 1][w & 2] + s_smaller[turn & 1][w | 1];      // ascending keys: the first k
      if (lo < hi) {
        hi = std::min(hi, lo + k * step);
        lo = k == 0 ? hi : lo + (k - 1) * step + 1;
      }
    }
    if ((threadIdx.x & 127) == 0) s_ends[w >> 1] = lo;
  }
  __syncthreads();
  int64_t lo = s_ends[0], hi = s_ends[1];
  if (hi - lo <= kHeld) {
    const int n_held = int(hi - lo);
#pragma unroll 8
    for (int i = threadIdx.x; i < n_held; i += 256) s_key[i] = keys[lo + i];
    __syncthreads();
    int a = 0, b = n_held;
    while (a < b) {
      const int mid = (a + b) >> 1;
      const bool below = int64_t(s_key[mid]) < g;
      a = below ? mid + 1 : a;
      b = below ? b : mid;
    }
    if (g <= groups) offsets[g] = lo + a;
    return;
  }
  if (g > groups) return;
  while (lo < hi) {
    const int64_t q = (hi - lo) >> 2, a = lo + q, b = a + q, c = b + q;      // lo <= a <= b <= c < hi
    const bool sa = int64_t(keys[a]) < g, sb = int64_t(keys[b]) < g, sc = int64_t(keys[c]) < g;
    lo = sc ? c + 1 : sb ? b + 1 : sa ? a + 1 : lo;
    hi = !sa ? a : !sb ? b : !sc ? c : hi;
  }
  offsets[g] = lo;
}

int key_bits(int64_t groups) {      // of a key in [0, groups]
  int b = 1;
  while ((groups >> b) != 0) ++b;
  return b;
}

struct SortSpace {
  uint32_t *counts, *totals, *keys;
  uint64_t* words[2];
  size_t bytes;
};

SortSpace sort_space(void* ws, int64_t n, int64_t groups) {
  const int64_t nb = (n + kBlockKeys - 1) / kBlockKeys;
  const int passes = (key_bits(groups) + kMaxBits - 1) / kMaxBits;
  char* p = static_cast<char*>(ws);
  SortSpace s{};
  auto take = [&](size_t bytes) {
    char* at = p + s.bytes;
    s.bytes += align_up(bytes, 256);
    return at;
  };
  if (n > kSmall) {
    const int digit = (key_bits(groups) + passes - 1) / passes;
    s.counts = reinterpret_cast<uint32_t*>(take((size_t(nb) * 4) << digit));
    s.totals = reinterpret_cast<uint32_t*>(take(size_t(4) << digit));
    for (int k = 0; k < std::min(passes - 1, 2); ++k) s.words[k] = reinterpret_cast<uint64_t*>(take(size_t(n) * 8));
  }
  if (n > kSmall ? passes > 1 : groups >= kSmallBounds) s.keys = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
  return s;
}

template <typename I, bool kFirst>
void pass(const Pass& p, hipStream_t st) {
  k_count<I, kFirst><<<p.nb, kT, 0, st>>>(p);
  if (p.totals != nullptr) k_scan<<<((1 << p.bits) + 63) / 64, 1024, 0, st>>>(p.counts, p.bits, p.nb, p.totals);
  k_place<I, kFirst><<<p.nb, kT, 0, st>>>(p);
}

template <typename I>
hipError_t sort(const SortArgs& a, void* ws, hipStream_t st) {
  const SortSpace s = sort_space(ws, a.n, a.groups);
  const int bits = key_bits(a.groups);
  const unsigned bounds = unsigned((a.groups + 256) / 256);
  if (a.n <= kSmall) {
    const int passes = (bits + kSmallBits - 1) / kSmallBits;
    if (a.n > 2048)
      k_sort_small<I, 1024, 8><<<1, 1024, 0, st>>>(a, bits, passes, s.keys);
    else if (a.n > 256)
      k_sort_small<I, 256, 8><<<1, 256, 0, st>>>(a, bits, passes, s.keys);
    else
      k_sort_small<I, 256, 1><<<1, 256, 0, st>>>(a, bits, passes, s.keys);
    if (s.keys != nullptr) k_bounds<<<bounds, 256, 0, st>>>(s.keys, a.n, a.groups, a.offsets);
    return hipGetLastError();
  }
  const int passes = (bits + kMaxBits - 1) / kMaxBits;
  Pass p{};
  p.src = a.ids;
  p.n = a.n;
  p.groups = uint32_t(a.groups);
  p.bits = (bits + passes - 1) / passes;
  p.nb = int((a.n + kBlockKeys - 1) / kBlockKeys);
  p.counts = s.counts;
  p.totals = p.nb <= kFewBlocks ? nullptr : s.totals;
  for (int k = 0; k < passes; ++k) {
    const bool last = k == passes - 1;
    p.shift = k * p.bits;
    p.out = last ? nullptr : s.words[k & 1];
    if (last) {
      p.out_keys = s.keys;
      p.order = a.order;
      p.place = a.place;
      p.offsets = passes == 1 ? a.offsets : nullptr;
    }
    k == 0 ? pass<I, true>(p, st) : pass<I, false>(p, st);
    p.src = p.out;
  }
  if (passes > 1) k_bounds<<<bounds, 256, 0, st>>>(s.keys, a.n, a.groups, a.offsets);
  return hipGetLastError();
}

}  // namespace

size_t group_sort_ws_bytes(int64_t n, int64_t groups) { return sort_space(nullptr, n, groups).bytes; }

hipError_t launch_group_sort(const SortArgs& a, void* ws, hipStream_t st) {
  return a.id_bytes == 4 ? sort<int32_t>(a, ws, st) : sort<int64_t>(a, ws, st);
}

}  // namespace gs
