// Many adapters beside one shared weight: what the plan, the products and the entry points share.
#pragma once

#include "dropout.h"
#include "internal.h"

namespace loftq {

constexpr int kTile = 64;          // tokens of a tile: of one slot each
constexpr int kMostSlots = 1024;

// Where the pieces of a plan lie (int32 words).  `order` and what lies before it are public.
struct PlanLayout {
  int64_t n;
  int slots;
  int64_t order;        // [n] tokens, slot after slot; a slot's in rising order
  int64_t info;         // tiles, chunks, n, slots
  int64_t tiles;        // [max_tiles][4]: slot (-1: no adapter), first place in `order`, tokens, 0
  int64_t rows;         // [max_tiles][kTile]: a tile's tokens, the slot's last one again past them
  int64_t chunks;       // [max_chunks][4]: slot, first tile, tiles, chunks of the slot; slots of several chunks come first
  int64_t slot_parts;   // [slots + 1]: chunks of such slots before a slot: where its own lie, if it is one
  int64_t slot_used;    // [slots + 1]: slots with tokens before a slot
  int64_t counts;       // [plan_wgs][slots + 1]: tokens by workgroup and slot (more than one workgroup)
  int64_t words;
  int64_t max_tiles, max_chunks;
  int64_t max_parts;    // chunks of the slots of several
  int chunk_tiles;      // tiles of a chunk (the last of a slot may have fewer)
  int wgs;
  int64_t per_wg;
};

constexpr int kPlanThreads = 512;

inline PlanLayout plan_layout(int64_t n, int slots) {
  PlanLayout p{};
  p.n = n;
  p.slots = slots;
  const int64_t groups = n < slots + 1 ? n : slots + 1, whole = n / kTile;
  // a group of c tokens has at most (c + 63) / 64 tiles, and those of q tiles (q + c - 1) / c chunks of c
  p.max_tiles = whole + groups;
  // about four chunks of a batch with one slot, of 2 to 128 tiles: with the groups of features they fill the CUs, and
  // most slots of a batch with several have one, whose sums need no second pass
  p.chunk_tiles = static_cast<int>(whole <= 8 ? 2 : (whole >= 512 ? 128 : (whole + 3) / 4));
  // whole / chunk_tiles, in a form that grows with n
  const int64_t full = whole / 128 > 4 ? whole / 128 : 4;
  // a slot of w whole tiles has at most w / chunk_tiles + 1 chunks: over all slots `full` and one for each slot
  p.max_chunks = full + groups;
  // with several of them w / chunk_tiles is 1 at least, so that the slots of several are no more than `full` either
  p.max_parts = n <= p.chunk_tiles * kTile ? 0 : full + (full < slots ? full : slots);
  p.per_wg = (n + 255) / 256;
  p.per_wg = p.per_wg < 4096 ? 4096 : (p.per_wg + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  p.wgs = static_cast<int>((n + p.per_wg - 1) / p.per_wg);
  auto pad = [](int64_t w) { return (w + 3) / 4 * 4; };
  p.order = pad(slots + 2);
  p.info = p.order + pad(n);
  p.tiles = p.info + 4;
  p.rows = p.tiles + 4 * p.max_tiles;
  p.chunks = p.rows + kTile * p.max_tiles;
  p.slot_parts = p.chunks + 4 * p.max_chunks;
  p.slot_used = p.slot_parts + pad(slots + 1);
  p.counts = p.slot_used + pad(slots + 1);
  p.words = p.counts + (p.wgs > 1 ? pad(static_cast<int64_t>(p.wgs) * (slots + 1)) : 0);
  return p;
}

hipError_t launch_adapters_plan(const int32_t* slot_of, int32_t* plan, const PlanLayout& p, hipStream_t s);

// What the kernels read of a plan.
struct PlanView {
  const int32_t* info;
  const int4* tiles;
  const int32_t* rows;
  const int4* chunks;
  const int32_t* slot_parts;
  const int32_t* slot_used;
  int32_t n, slots, max_tiles, max_chunks, max_parts;
};
inline PlanView plan_view(const int32_t* plan, const PlanLayout& p) {
  return PlanView{plan + p.info, reinterpret_cast<const int4*>(plan + p.tiles), plan + p.rows,
                  reinterpret_cast<const int4*>(plan + p.chunks), plan + p.slot_parts, plan + p.slot_used, static_cast<int32_t>(p.n),
                  static_cast<int32_t>(p.slots), static_cast<int32_t>(p.max_tiles), static_cast<int32_t>(p.max_chunks),
                  static_cast<int32_t>(p.max_parts)};
}

// A pool of adapters: `ranks` and `gains` may be null.
struct Pool {
  const void *B, *A;
  loftq_dtype_t dt;
  int slots, rank, rp;   // rp: the rank in whole 16s
  const int32_t* ranks;
  const float* gains;
  float gain;            // alpha times dropout's scale
};

// Slots with tokens that a batch may have: the slots of the factors' prepared forms.
inline int64_t used_slots(int64_t n, int slots) { return n < slots ? n : slots; }

// Forms of a pool's factors in bf16 that the products read, for the slots with tokens, one after another.  Ranks
// past a slot's own are zeros.  Null where not wanted.
struct Prepare {
  __bf16* Bp;      // [used][rows][rp]
  __bf16* Bt;      // [used][rp][rows8]: zeros past `rows`
  __bf16* Ab;      // [used][rp][cols]
  __bf16* At;      // [used][cols][rp]
  float *dB, *dA;  // gradients, or null: zeros for the slots without tokens
  int64_t rows, rows8, cols;
  unsigned wgs;    // a slot's workgroups, set by the launcher
};
hipError_t launch_adapters_prepare(Prepare p, const PlanView& plan, const Pool& pool, hipStream_t s);

// P = keep(L) F^T over the tokens of each tile, as partial sums over `ks` K ranges [ks][max_tiles 64][rp].  L has K
// columns (8 | K), F a row of K elements for each rank, slot after slot.
struct AdapterDown {
  const __bf16* L;       // null: no such job
  int64_t K;
  const void* F;         // of the launch's type
  int64_t slot_elems;    // elements from slot to slot
  bool prepared;         // one of Prepare's forms: its slots are the ones with tokens
  float* out;
  int ks;
  unsigned wgs;          // set by the launcher
  DropArg drop;
};
int adapters_down_splits(int64_t n, int slots, int64_t K, int rp);
// at least the partials of every call of up to n tokens and of rank up to rp
int64_t adapters_down_floats_bound(int64_t n, int slots, int64_t K, int rp);
struct AdapterDownJobs {
  AdapterDown job[2];
};
// with the forms of `prepare` in the same launch (they are for the launch after it)
hipError_t launch_adapters_down(AdapterDownJobs jobs, loftq_dtype_t factor, const Prepare& prepare, const PlanView& plan,
                                const Pool& pool, hipStream_t s);

// The partials in range order: their sum (fp32, [max_tiles 64][rp]) and as three bf16 pieces rank-major
// [3][rp][max_tiles 64], zeros past a tile's tokens.  Either may be null.
struct AdapterSum {
  const float* partials;   // null: no such job
  int ks;
  float* sum;
  __bf16* St;
};
struct AdapterSumJobs {
  AdapterSum job[2];
};
// with the forms of `prepare` in the same launch
hipError_t launch_adapters_sum(AdapterSumJobs jobs, const Prepare& prepare, const PlanView& plan, const Pool& pool, hipStream_t s);

// out = in + gain keep(H F^T): H the partial sums of `ks` ranges, F [slot][features][ld] in bf16.
struct AdapterUp {
  const float* H;
  int ks;
  int64_t features;
  const __bf16* F;
  int64_t ld;            // 8 | ld
  bool prepared;
  const void* in;        // or null
  void* out;
  loftq_dtype_t odt;
  DropArg drop;          // thr != 0: 4 | features
};
hipError_t launch_adapters_up(const AdapterUp& u, const PlanView& plan, const Pool& pool, hipStream_t s);

// The gradients of the factors over the tokens of each chunk: job 0 dB (over dY's columns, F = nf in whole 8s), job 1 dA.
// A slot of one chunk is written to `out` at once, the partial sums of more to `partials` [max_parts][F rp].
struct AdapterGrad {
  const __bf16 *L, *St;
  float *partials, *out;
  int64_t F, nf;
  DropArg drop;
};
struct AdapterGradJobs {
  AdapterGrad job[2];
};
hipError_t launch_adapters_grad(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s);
// the sums of partials; zeros for a batch without tokens
hipError_t launch_adapters_grad_sum(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s);

// dY in rows of `to` columns, zeros past `from`
hipError_t launch_adapters_pad(const __bf16* in, __bf16* out, int64_t n, int64_t from, int64_t to, hipStream_t s);

}  // namespace loftq
