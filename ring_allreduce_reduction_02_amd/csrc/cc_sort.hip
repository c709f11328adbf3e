// Stable sort of small integer keys with their positions: the rows of one
// expert, or of one word of a vocabulary, brought together in the order they
// came in.
//
// Least significant digit first, 8 bits a pass.  A pass is three kernels: the
// digit counts of every tile, their exclusive prefix in (digit, tile) order,
// and the scatter, in which a key's place inside its tile is the number of
// equal digits before it: in its wave's earlier rounds, in the lanes below it
// (one ballot per bit), and in the waves before it.  Every place is a count,
// so nothing depends on the order in which workgroups run.  One pass over 8
// ranks x 32768 keys takes 4, 3.5 and 5 us, bound by latency.

#include <algorithm>

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

constexpr int kSortBlock = 256;
constexpr int kSortWaves = kSortBlock / 64;
constexpr int kSortRounds = 4;                              // keys per lane
constexpr int kSortTile = kSortBlock * kSortRounds;         // 1024 keys
constexpr int kDigits = 256;

struct SortArgs {
  const char* keys;      // first pass: the caller's keys
  uint64_t key_stride;
  const int* kin;        // later passes
  const int* vin;
  int* kout;
  int* vout;
  char* order;
  uint64_t os;
  char* counts;          // set: the pass gives positions and counts
  uint64_t cs;
  uint32_t* hist;        // [N][kDigits][tiles]
  uint64_t n;
  uint32_t nkeys;
  uint32_t tiles;
  int shift;
  int first;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint64_t rank, uint64_t i) {
  if (!a.first) return (uint32_t)a.kin[rank * a.n + i];
  const uint32_t k = (uint32_t)((const int*)(a.keys + rank * a.key_stride))[i];
  return k < a.nkeys ? k : a.nkeys;
}

// The lanes of a wave whose digit is d, for every lane of `in`.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool in) {
  uint64_t same = __ballot(in);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint64_t one = __ballot((d >> b) & 1u);
    same &= ((d >> b) & 1u) ? one : ~one;
  }
  return same;
}

// Up to kLdsSortMax keys of a rank, all passes in one workgroup: keys and
// positions stay in registers between passes and change places through LDS.
// Wave w holds the keys [w, w + 1) * 64 R, 64 a round, as in a tile below.
// 4096 keys of 15 bits on each of 8 ranks: 11.5 us in one launch; the six
// launches of two passes over tiles took about 30.
constexpr int kLdsSortBlock = 1024;
constexpr int kLdsSortWaves = kLdsSortBlock / 64;
constexpr int kLdsSortMax = 8192;

template <int R>
__global__ __launch_bounds__(kLdsSortBlock) void k_sort_lds(SortArgs a, int passes) {
  __shared__ uint32_t cnt[kLdsSortWaves][kDigits];
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t wsum[kDigits / 64];
  __shared__ uint2 kv[R * kLdsSortBlock];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t n = (uint32_t)a.n, i0 = wave * 64 * R + lane;
  const uint64_t rank = blockIdx.x, below = (1ull << lane) - 1;
  uint32_t key[R], val[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const uint32_t i = i0 + q * 64;
    key[q] = i < n ? sort_key(a, rank, i) : 0u;
    val[q] = i;
  }
  for (int pass = 0; pass < passes; ++pass) {
    for (int d = threadIdx.x; d < kLdsSortWaves * kDigits; d += kLdsSortBlock) (&cnt[0][0])[d] = 0;
    __syncthreads();
    uint32_t place[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool in = i0 + q * 64 < n;
      const uint32_t d = (key[q] >> (8 * pass)) & (kDigits - 1);
      const uint64_t same = same_digit(d, in);
      volatile uint32_t* c = &cnt[wave][d];
      const uint32_t before = *c;
      place[q] = before + (uint32_t)__popcll(same & below);
      if (in && (same & below) == 0) *c = before + (uint32_t)__popcll(same);
    }
    __syncthreads();
    // exclusive prefix over (digit, wave)
    if (threadIdx.x < kDigits) {
      uint32_t all = 0;
#pragma unroll
      for (int w = 0; w < kLdsSortWaves; ++w) {
        const uint32_t c = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = all;
        all += c;
      }
      uint32_t s = all;
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t t = __shfl_up(s, d);
        if (lane >= d) s += t;
      }
      base[threadIdx.x] = s - all;
      if (lane == 63) wsum[wave] = s;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (i0 + q * 64 >= n) continue;
      const uint32_t d = (key[q] >> (8 * pass)) & (kDigits - 1);
      uint32_t at = base[d] + cnt[wave][d] + place[q];
      for (uint32_t w = 0; w < (d >> 6); ++w) at += wsum[w];
      kv[at] = make_uint2(key[q], val[q]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t i = i0 + q * 64;
      if (i >= n) continue;
      key[q] = kv[i].x;
      val[q] = kv[i].y;
    }
  }
  if (a.counts) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t i = i0 + q * 64;
      if (i < n) ((int*)(a.order + rank * a.os))[i] = key[q] < a.nkeys ? (int)val[q] : -1;
    }
    for (uint32_t e = threadIdx.x; e < a.nkeys; e += kLdsSortBlock) {
      uint32_t b[2];
      for (int s = 0; s < 2; ++s) {   // first sorted place of the key e + s
        uint32_t lo = 0, hi = n;
        while (lo < hi) {
          const uint32_t mid = (lo + hi) >> 1;
          if (kv[mid].x < e + s) lo = mid + 1; else hi = mid;
        }
        b[s] = lo;
      }
      ((int*)(a.counts + rank * a.cs))[e] = (int)(b[1] - b[0]);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const uint32_t i = i0 + q * 64;
    if (i >= n) continue;
    a.kout[rank * a.n + i] = (int)key[q];
    a.vout[rank * a.n + i] = (int)val[q];
  }
}

__global__ __launch_bounds__(kSortBlock) void k_sort_hist(SortArgs a) {
  __shared__ uint32_t h[kDigits];
  h[threadIdx.x] = 0;
  __syncthreads();
  const uint64_t i0 = (uint64_t)blockIdx.x * kSortTile;
  for (int q = 0; q < kSortRounds; ++q) {
    const uint64_t i = i0 + (uint64_t)q * kSortBlock + threadIdx.x;
    if (i < a.n) atomicAdd(&h[(sort_key(a, blockIdx.y, i) >> a.shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
  a.hist[((uint64_t)blockIdx.y * kDigits + threadIdx.x) * a.tiles + blockIdx.x] = h[threadIdx.x];
}

// Exclusive prefix over a rank's kDigits * tiles counts, in place, 8 of them a
// thread.  (tiles * kDigits is a multiple of 8.)
constexpr int kScanBlock = 1024;
constexpr int kScanEach = 8;
__global__ __launch_bounds__(kScanBlock) void k_sort_scan(uint32_t* hist, uint64_t count) {
  __shared__ uint32_t wsum[kScanBlock / 64];
  uint32_t* h = hist + (uint64_t)blockIdx.x * count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t carry = 0;
  for (uint64_t b = 0; b < count; b += kScanBlock * kScanEach) {
    const uint64_t i = b + (uint64_t)threadIdx.x * kScanEach;
    uint32_t v[kScanEach] = {}, own = 0;
    if (i < count) {
      const u32x4 lo = *(const u32x4*)(h + i), hi = *(const u32x4*)(h + i + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = lo[k];
        v[4 + k] = hi[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kScanEach; ++k) own += v[k];
    uint32_t s = own;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t t = __shfl_up(s, d);
      if (lane >= d) s += t;
    }
    __syncthreads();   // the last round's wsum is read
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    uint32_t at = carry + s - own;
    for (int w = 0; w < kScanBlock / 64; ++w) {
      if (w < wave) at += wsum[w];
      carry += wsum[w];
    }
    if (i < count) {
      u32x4 lo, hi;
#pragma unroll
      for (int k = 0; k < kScanEach; ++k) {
        if (k < 4) lo[k] = at; else hi[k - 4] = at;
        at += v[k];
      }
      *(u32x4*)(h + i) = lo;
      *(u32x4*)(h + i + 4) = hi;
    }
  }
}

// Positions and counts from sorted keys (more than one pass of tiles).
__global__ __launch_bounds__(kSortBlock) void k_sort_order(SortArgs a) {
  const uint64_t r = blockIdx.y, i = (uint64_t)blockIdx.x * kSortBlock + threadIdx.x;
  const int* keys = a.kin + r * a.n;
  if (i < a.n) ((int*)(a.order + r * a.os))[i] = (uint32_t)keys[i] < a.nkeys ? a.vin[r * a.n + i] : -1;
  if (i < a.nkeys) {
    uint64_t b[2];
    for (int s = 0; s < 2; ++s) {
      uint64_t lo = 0, hi = a.n;
      while (lo < hi) {
        const uint64_t mid = (lo + hi) >> 1;
        if ((uint64_t)keys[mid] < i + s) lo = mid + 1; else hi = mid;
      }
      b[s] = lo;
    }
    ((int*)(a.counts + r * a.cs))[i] = (int)(b[1] - b[0]);
  }
}

__global__ __launch_bounds__(kSortBlock) void k_sort_scatter(SortArgs a) {
  __shared__ uint32_t cnt[kSortWaves][kDigits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int d = threadIdx.x; d < kSortWaves * kDigits; d += kSortBlock) (&cnt[0][0])[d] = 0;
  __syncthreads();
  // wave w holds the tile's keys [w, w + 1) * 64 * rounds, 64 a round
  const uint64_t i0 = (uint64_t)blockIdx.x * kSortTile + (uint64_t)wave * 64 * kSortRounds;
  uint32_t key[kSortRounds], place[kSortRounds];
  int val[kSortRounds];
  const uint64_t below = (1ull << lane) - 1;
  for (int q = 0; q < kSortRounds; ++q) {
    const uint64_t i = i0 + (uint64_t)q * 64 + lane;
    const bool in = i < a.n;
    key[q] = in ? sort_key(a, blockIdx.y, i) : 0u;
    val[q] = in ? (a.first ? (int)i : a.vin[(uint64_t)blockIdx.y * a.n + i]) : 0;
    const uint32_t d = (key[q] >> a.shift) & (kDigits - 1);
    const uint64_t same = same_digit(d, in);
    // lanes of one digit read its count, then the lowest of them adds theirs
    // (a wave's LDS accesses complete in program order; volatile keeps it)
    volatile uint32_t* c = &cnt[wave][d];
    const uint32_t before = *c;
    place[q] = before + (uint32_t)__popcll(same & below);
    if (in && (same & below) == 0) *c = before + (uint32_t)__popcll(same);
  }
  __syncthreads();
  {
    const int d = threadIdx.x;   // kSortBlock == kDigits
    const uint32_t* first = a.hist + ((uint64_t)blockIdx.y * kDigits + d) * a.tiles;
    uint32_t at = first[blockIdx.x];
    // one pass: a digit is a key, and nkeys < kDigits of them have a next one
    if (a.counts && blockIdx.x == 0 && (uint32_t)d < a.nkeys)
      ((int*)(a.counts + (uint64_t)blockIdx.y * a.cs))[d] = (int)(first[a.tiles] - first[0]);
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = cnt[w][d];
      cnt[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int q = 0; q < kSortRounds; ++q) {
    const uint64_t i = i0 + (uint64_t)q * 64 + lane;
    if (i >= a.n) continue;
    const uint32_t d = (key[q] >> a.shift) & (kDigits - 1);
    const uint64_t to = cnt[wave][d] + place[q];
    if (a.counts) {
      ((int*)(a.order + (uint64_t)blockIdx.y * a.os))[to] = key[q] < a.nkeys ? val[q] : -1;
    } else {
      a.kout[(uint64_t)blockIdx.y * a.n + to] = (int)key[q];
      a.vout[(uint64_t)blockIdx.y * a.n + to] = val[q];
    }
  }
}

uint64_t up(uint64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

SortPlan sort_plan(int N, uint64_t n, uint32_t nkeys) {
  SortPlan p;
  p.N = N;
  p.n = n;
  p.nkeys = nkeys;
  p.passes = 1;
  while (p.passes < 4 && (nkeys >> (8 * p.passes)) != 0) ++p.passes;   // the key nkeys itself is sorted too
  p.tiles = n <= kLdsSortMax ? 0 : (n + kSortTile - 1) / kSortTile;
  const uint64_t arr = up((uint64_t)N * n * 4);
  p.bytes = (p.tiles && p.passes > 1 ? 4 : 2) * arr + up((uint64_t)N * kDigits * p.tiles * 4);
  return p;
}

hipError_t launch_sort(SortLaunch* L) {
  const SortPlan& p = L->p;
  const uint64_t arr = up((uint64_t)p.N * p.n * 4);
  SortArgs a = {};
  a.keys = L->keys; a.key_stride = L->key_stride;
  a.n = p.n; a.nkeys = p.nkeys;
  a.order = L->order; a.os = L->order_stride; a.cs = L->counts_stride;
  if (p.n == 0 || p.tiles == 0) {
    a.counts = L->counts;
    a.first = 1;
    a.kout = (int*)L->ws;
    a.vout = (int*)(L->ws + arr);
    const dim3 grid((unsigned)p.N), blk(kLdsSortBlock);
    if (p.n <= 1024) CC_LAUNCH(k_sort_lds<1>, grid, blk, 0, L->st, a, p.passes);
    else if (p.n <= 2048) CC_LAUNCH(k_sort_lds<2>, grid, blk, 0, L->st, a, p.passes);
    else if (p.n <= 4096) CC_LAUNCH(k_sort_lds<4>, grid, blk, 0, L->st, a, p.passes);
    else CC_LAUNCH(k_sort_lds<8>, grid, blk, 0, L->st, a, p.passes);
    L->sorted_keys = a.kout;
    L->sorted_vals = a.vout;
    return hipGetLastError();
  }
  const int two = p.passes > 1;
  int* k[2] = {(int*)L->ws, (int*)(L->ws + 2 * two * arr)};
  int* v[2] = {(int*)(L->ws + arr), (int*)(L->ws + 3 * two * arr)};
  a.hist = (uint32_t*)(L->ws + (two ? 4 : 2) * arr);
  a.tiles = (uint32_t)p.tiles;
  const dim3 grid((unsigned)p.tiles, (unsigned)p.N), blk(kSortBlock);
  for (int pass = 0; pass < p.passes; ++pass) {
    a.first = pass == 0;
    a.shift = 8 * pass;
    a.kin = k[(pass + 1) & 1]; a.vin = v[(pass + 1) & 1];
    a.kout = k[pass & 1]; a.vout = v[pass & 1];
    a.counts = p.passes == 1 ? L->counts : nullptr;
    CC_LAUNCH(k_sort_hist, grid, blk, 0, L->st, a);
    CC_LAUNCH(k_sort_scan, dim3((unsigned)p.N), dim3(kScanBlock), 0, L->st, a.hist, (uint64_t)kDigits * p.tiles);
    CC_LAUNCH(k_sort_scatter, grid, blk, 0, L->st, a);
  }
  L->sorted_keys = k[(p.passes - 1) & 1];
  L->sorted_vals = v[(p.passes - 1) & 1];
  if (L->counts && p.passes > 1) {
    a.counts = L->counts;
    a.kin = L->sorted_keys;
    a.vin = L->sorted_vals;
    const uint64_t m = std::max<uint64_t>(p.n, p.nkeys);
    CC_LAUNCH(k_sort_order, dim3((unsigned)((m + kSortBlock - 1) / kSortBlock), (unsigned)p.N), blk, 0, L->st, a);
  }
  return hipGetLastError();
}

}  // namespace cc
