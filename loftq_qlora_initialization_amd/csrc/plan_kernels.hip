// The plan of a batch: a stable counting sort of its tokens by slot, and the tiles and chunks
// that the products divide their work by.  Stable without atomics on the order: a wave owns
// consecutive tokens, its own counters, and ranks 64 of them at a time by ballots over the
// bits of their slots.
//
// Bound by latency: 64 tokens are one workgroup's few dependent steps (5.0 us with the launch), 65536 of 512 slots two
// launches of 16 workgroups (22 us), whose waves load eight tokens a lane at once (32 us with a load for each step).
#include "adapters.h"

namespace loftq {
namespace {

constexpr int kWaves = kPlanThreads / 64;

// The slots of kAhead tokens, `stride` apart from i0 on, with all loads in flight at once; kNone at `end` and past it.
constexpr int kAhead = 8, kNone = kMostSlots + 1;
__device__ __forceinline__ void groups_of(const int32_t* slot_of, int64_t i0, int stride, int64_t end, int slots, int (&g)[kAhead]) {
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    const int64_t i = i0 + e * stride;
    g[e] = slot_of[i < end ? i : end - 1];
  }
#pragma unroll
  for (int e = 0; e < kAhead; ++e) {
    const int in = static_cast<unsigned>(g[e]) < static_cast<unsigned>(slots) ? g[e] : slots;
    g[e] = i0 + e * stride < end ? in : kNone;
  }
}

// tokens by slot of a workgroup's share
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const int32_t* __restrict__ slot_of, PlanLayout p,
                                                                  int32_t* __restrict__ plan) {
  __shared__ int hist[kMostSlots + 1];
  for (int s = threadIdx.x; s <= p.slots; s += kPlanThreads) hist[s] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * p.per_wg, end = begin + p.per_wg < p.n ? begin + p.per_wg : p.n;
  for (int64_t i = begin; i < end; i += kAhead * kPlanThreads) {
    int g[kAhead];
    groups_of(slot_of, i + threadIdx.x, kPlanThreads, end, p.slots, g);
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (g[e] != kNone) atomicAdd(&hist[g[e]], 1);
  }
  __syncthreads();
  for (int s = threadIdx.x; s <= p.slots; s += kPlanThreads)
    plan[p.counts + static_cast<int64_t>(blockIdx.x) * (p.slots + 1) + s] = hist[s];
}

struct Sums {
  int tokens, tiles;
  int parts;   // chunks of the slots of several
  int slots;   // slots with tokens, and in the high half those of them of one chunk: one exchange less than with a number each
};
constexpr int kOne = 1 << 16;
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return Sums{a.tokens + b.tokens, a.tiles + b.tiles, a.parts + b.parts, a.slots + b.slots};
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const int32_t* __restrict__ slot_of, PlanLayout p,
                                                                  int32_t* __restrict__ plan) {
  __shared__ int count[kWaves][kMostSlots + 1];   // a wave's tokens by slot, then the place of its next one
  __shared__ Sums first[kMostSlots + 2];         // what lies before a slot
  __shared__ Sums wave_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, groups = p.slots + 1;
  for (int s = lane; s < groups; s += 64) count[w][s] = 0;
  __syncthreads();
  const int64_t per_wave = p.per_wg / kWaves;
  const int64_t begin = blockIdx.x * p.per_wg + w * per_wave, end = begin + per_wave < p.n ? begin + per_wave : p.n;
  for (int64_t i = begin; i < end; i += kAhead * 64) {
    int g[kAhead];
    groups_of(slot_of, i + lane, 64, end, p.slots, g);
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (g[e] != kNone) atomicAdd(&count[w][g[e]], 1);
  }
  __syncthreads();
  // a slot's total, and the place of each wave's first token among the slot's
  const int each = (groups + kPlanThreads - 1) / kPlanThreads, s0 = tid * each;
  Sums mine{0, 0, 0, 0};
  for (int s = s0; s < s0 + each && s < groups; ++s) {
    int before = 0, total = 0;
    if (p.wgs > 1)
#pragma unroll 8
      for (int b = 0; b < p.wgs; ++b) {
        const int c = plan[p.counts + static_cast<int64_t>(b) * groups + s];
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
        total += c;
      }
    for (int v = 0; v < kWaves; ++v) {
      const int c = count[v][s];
      count[v][s] = before;
      before += c;
    }
    if (p.wgs == 1) total = before;
    const int tiles = (total + kTile - 1) / kTile, chunks = s < p.slots ? (tiles + p.chunk_tiles - 1) / p.chunk_tiles : 0;
    const Sums own{total, tiles, chunks > 1 ? chunks : 0, chunks > 1 ? 1 : (chunks == 1 ? 1 + kOne : 0)};
    first[s] = mine;     // within the thread, made whole below
    mine = mine + own;
  }
  Sums upto = mine;     // sums over the wave's lanes up to this one
  for (int d = 1; d < 64; d <<= 1) {
    const Sums o{__shfl_up(upto.tokens, d), __shfl_up(upto.tiles, d), __shfl_up(upto.parts, d), __shfl_up(upto.slots, d)};
    if (lane >= d) upto = upto + o;
  }
  if (lane == 63) wave_sum[w] = upto;
  __syncthreads();
  Sums base{upto.tokens - mine.tokens, upto.tiles - mine.tiles, upto.parts - mine.parts, upto.slots - mine.slots};
  for (int v = 0; v < w; ++v) base = base + wave_sum[v];
  for (int s = s0; s < s0 + each && s < groups; ++s) first[s] = first[s] + base;
  if (tid == 0) {
    Sums all{0, 0, 0, 0};
    for (int v = 0; v < kWaves; ++v) all = all + wave_sum[v];
    first[groups] = all;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int s = tid; s <= groups; s += kPlanThreads) plan[s] = first[s].tokens;
    for (int s = tid; s < groups; s += kPlanThreads) {
      plan[p.slot_parts + s] = first[s].parts;
      plan[p.slot_used + s] = first[s].slots & (kOne - 1);
    }
    if (tid == 0)
      *reinterpret_cast<int4*>(plan + p.info) =
          make_int4(first[groups].tiles, first[groups].parts + (first[groups].slots >> 16), static_cast<int>(p.n), p.slots);
  }
  const int parts = first[groups].parts;
  volatile int* next = count[w];
  auto place = [&](int64_t i, int g) __attribute__((always_inline)) {
    const bool live = g != kNone;
    // the lanes with this lane's slot
    uint64_t peers = ~0ull;
#pragma unroll
    for (int b = 0; b < 11; ++b) {
      const uint64_t set = __ballot((g >> b) & 1);
      peers &= (g >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    const int from = live ? next[g] : 0;
    __builtin_amdgcn_wave_barrier();   // every lane has read before the last of its peers writes
    if (live && (peers >> lane) == 1ull) next[g] = from + rank + 1;
    __builtin_amdgcn_wave_barrier();
    if (!live) return;
    const int k = from + rank, total = first[g + 1].tokens - first[g].tokens;   // the k-th of its slot
    const int tile = first[g].tiles + k / kTile, at = first[g].tokens + k;
    plan[p.order + at] = static_cast<int>(i);
    int32_t* rows = plan + p.rows + static_cast<int64_t>(tile) * kTile;
    rows[k % kTile] = static_cast<int>(i);
    if (k % kTile == 0) {
      const int left = total - k;
      reinterpret_cast<int4*>(plan + p.tiles)[tile] = make_int4(g < p.slots ? g : -1, at, left < kTile ? left : kTile, 0);
      const int index = k / kTile, tiles = (total + kTile - 1) / kTile;
      if (g < p.slots && index % p.chunk_tiles == 0) {   // slots of several chunks come first
        const int at_chunk = tiles > p.chunk_tiles ? first[g].parts + index / p.chunk_tiles : parts + (first[g].slots >> 16);
        reinterpret_cast<int4*>(plan + p.chunks)[at_chunk] =
            make_int4(g, tile, tiles - index < p.chunk_tiles ? tiles - index : p.chunk_tiles,
                      (tiles + p.chunk_tiles - 1) / p.chunk_tiles);
      }
    }
    if (k == total - 1) {
      // to the tile's end, four at once: many slots end in the last workgroup's tokens (65536 tokens of 512 slots: 29 us one
      // by one, 21 with this; the wave's lanes together, a slot at a time: 21 too, and 64 tokens of 48 slots 8.8 instead of 5.1)
      int j = k % kTile + 1;
      const int token = static_cast<int>(i);
      for (; j % 4 != 0; ++j) rows[j] = token;
      for (; j < kTile; j += 4) *reinterpret_cast<int4*>(rows + j) = make_int4(token, token, token, token);
    }
  };
  for (int64_t i0 = begin; i0 < end; i0 += kAhead * 64) {
    int g[kAhead];
    groups_of(slot_of, i0 + lane, 64, end, p.slots, g);
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (i0 + e * 64 < end) place(i0 + e * 64 + lane, g[e]);   // the whole wave
  }
}

// without tokens
__global__ void plan_empty_kernel(PlanLayout p, int32_t* __restrict__ plan) {
  for (int s = threadIdx.x; s < p.slots + 2; s += blockDim.x) plan[s] = 0;
  for (int s = threadIdx.x; s < p.slots + 1; s += blockDim.x) plan[p.slot_parts + s] = plan[p.slot_used + s] = 0;
  if (threadIdx.x == 0) *reinterpret_cast<int4*>(plan + p.info) = make_int4(0, 0, 0, p.slots);
}

}  // namespace

hipError_t launch_adapters_plan(const int32_t* slot_of, int32_t* plan, const PlanLayout& p, hipStream_t s) {
  if (p.n == 0) {
    LQ_LAUNCH("adapters_plan", plan_empty_kernel, dim3(1), dim3(256), 0, s, p, plan);
    return hipGetLastError();
  }
  if (p.wgs > 1)
    LQ_LAUNCH("adapters_plan_count", plan_count_kernel, dim3(p.wgs), dim3(kPlanThreads), 0, s, slot_of, p, plan);
  LQ_LAUNCH("adapters_plan", plan_place_kernel, dim3(p.wgs), dim3(kPlanThreads), 0, s, slot_of, p, plan);
  return hipGetLastError();
}

}  // namespace loftq
