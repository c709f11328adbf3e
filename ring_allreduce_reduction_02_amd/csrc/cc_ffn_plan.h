// Device code of the plan that the experts' grouped products run by: the
// experts' first compact rows, their row tiles of each size and the rows' places
// in their rank's buffer.  The host sums the kept rows of every (expert, source); a
// kernel of E workgroups (times any number of parts) writes the tables and may
// take the rows on the way.
#pragma once

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {

// Words an expert: its first compact row, its first row tile of each size, its
// kept rows from each source.  (Summed on the device instead, from counts in the
// launch's arguments, which lie in the host's memory, the plan alone took 4-7 us,
// and 12 with the rows of a decoding step.)
constexpr int kPlanHead = 1 + kFfnTiles;
constexpr int kPlanWords = 896;   // that fit a launch's arguments
struct PlanArgs {
  uint32_t v[kPlanWords];
  const uint32_t* w;      // in memory, or NULL: v
  int N, E;
  uint64_t cap;
  int* start;
  int2* mtab[kFfnTiles];
  int* rowmap;
};
// the arguments, and (many words) the launches that put them into memory
hipError_t ffn_plan_args(const FfnShape& s, const FfnWs& o, char* ws, const uint32_t* kept, hipStream_t st, PlanArgs* a);

namespace {

constexpr int kPlanBlock = 256;

__device__ __forceinline__ const uint32_t* plan_of(const PlanArgs& a, int e) {
  return (a.w ? a.w : a.v) + (uint64_t)e * (kPlanHead + a.N);
}

// Expert e's row tiles and first compact row, by a workgroup.
__device__ __forceinline__ void plan_tables(const PlanArgs& a, int e) {
  const uint32_t* w = plan_of(a, e);
  const uint32_t r0 = w[0];
  uint32_t n = 0;
  for (int i = 0; i < a.N; ++i) n += w[kPlanHead + i];
#pragma unroll
  for (int k = 0; k < kFfnTiles; ++k)
    for (uint32_t t = threadIdx.x; t < (n + kFfnTile[k] - 1) / kFfnTile[k]; t += kPlanBlock)
      a.mtab[k][w[1 + k] + t] = make_int2(e, (int)(r0 + t * kFfnTile[k]));
  if (threadIdx.x == 0) {
    a.start[e] = (int)r0;
    if (e == a.E - 1) a.start[a.E] = (int)(r0 + n);
  }
}

// f(compact row, place in the rank's buffer) for every `step`-th kept row of
// expert e from its `first` on, both the same on all lanes of a wave.  The words
// lie in the host's memory: a lane reads its source's, all at once.
template <class F>
__device__ __forceinline__ void plan_rows(const PlanArgs& a, int e, uint32_t first, uint32_t step, F f) {
  static_assert(kMaxRanks <= 64, "a source a lane");
  const uint32_t* w = plan_of(a, e);
  const int lane = threadIdx.x & 63, per = a.E / a.N;
  uint32_t incl = lane < a.N ? w[kPlanHead + lane] : 0;
  const uint32_t r0 = w[0];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)incl, d);
    if (lane >= d) incl += o;
  }
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  for (uint32_t l = first; l < total; l += step) {
    const int i = __builtin_popcountll(__ballot(incl <= l));   // the first source past l, for l < total
    const uint32_t before = i ? (uint32_t)__shfl((int)incl, i - 1) : 0;
    f(r0 + l, (uint32_t)(((uint64_t)i * per + e % per) * a.cap) + (l - before));
  }
}

// The same where the tables are written: four workgroups' worth of waves, a row a
// wave, for 16 of a tile's 64 rows.  f(compact row, place, expert).
constexpr int kTileParts = 16;
template <class F>
__device__ __forceinline__ void table_rows(const int* start, const int2* mtab, const int* map, F f) {
  const int2 at = mtab[blockIdx.x];
  const int l = at.y + (int)blockIdx.y * (kFfnTile[kFfnTiles - 1] / kTileParts) +
                __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (l < start[at.x + 1]) f((uint32_t)l, (uint32_t)map[l], at.x);
}
static_assert(kFfnTile[kFfnTiles - 1] == 4 * kTileParts, "a row a wave");

// Whether one kernel makes the plan and takes the rows, E times (most / 4)
// workgroups: while all of them run at once.  @@RULE@@
inline unsigned plan_parts(const FfnShape& s) {
  const uint64_t parts = (s.most + 3) / 4;
  return parts * s.E <= 2048 ? (unsigned)(parts < 1 ? 1 : parts) : 0;
}

}  // namespace
}  // namespace cc
