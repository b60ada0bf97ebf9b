// Products of many adapters beside one shared weight: each token with the factors of its own slot.
//
// The plan has sorted the tokens into tiles of one slot each, so a tile's products are dense; its
// rows are gathered from X and scattered to Y by token number, whole rows at a time.  All of it
// is bound by loads and stores: X, Y0 and Y once each, a slot's factors once for every tile that
// shares a CU's or an XCD's cache.
#include "adapters.h"
#include "buffer.h"
#include "thin.h"

#include <type_traits>

namespace loftq {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kNowhere = 0x7FFFFFFFu;   // an offset past every resource, also with a row's length added: loads give zeros

// A tile of a plan that belongs to this call's sizes; slot -1 has no adapter, -2 is no tile.
struct TileInfo {
  int slot, count;
};
__device__ __forceinline__ TileInfo tile_info(const PlanView& p, int tile) {
  const int4 info = *reinterpret_cast<const int4*>(p.info), t = p.tiles[tile];   // neither load waits for the other
  const bool ours = info.z == p.n && info.w == p.slots && tile < info.x && t.x < p.slots;
  const int count = t.z < 0 ? 0 : (t.z > kTile ? kTile : t.z);
  return TileInfo{__builtin_amdgcn_readfirstlane(ours ? t.x : -2), __builtin_amdgcn_readfirstlane(ours ? count : 0)};
}
__device__ __forceinline__ int64_t token_at(const PlanView& p, int64_t place) {
  const int t = p.rows[place];
  return static_cast<unsigned>(t) < static_cast<unsigned>(p.n) ? t : 0;
}
__device__ __forceinline__ int slot_rank(const Pool& pool, int slot) {
  if (pool.ranks == nullptr) return pool.rank;
  const int r = pool.ranks[slot];
  return r < 0 ? 0 : (r > pool.rank ? pool.rank : r);
}

// The place of a slot among those with tokens.
__device__ __forceinline__ int64_t used_place(const PlanView& p, int slot) {
  const int u = p.slot_used[slot];
  return u < 0 ? 0 : (u < p.slots ? (u < p.n ? u : p.n - 1) : 0);
}

constexpr int kThreads = 256, kDownThreads = 512, kDownWaves = kDownThreads / 64;

// ---- the factors' forms for the products, eight elements a thread ----
// Element j of the eight from p on, `stride` elements apart, zero where j >= live: every load in flight at once.  A
// slot's factors, and a row of them, begin at any element where rows, rank or their product are odd, so it is the address
// itself that allows 16-byte loads.
template <typename T>
__device__ __forceinline__ bf16x8 pool_eight(const T* p, int64_t stride, int live) {
  T x[8];
  if (stride == 1 && live >= 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    typedef T piece_t __attribute__((ext_vector_type(kPer)));
#pragma unroll
    for (int c = 0; c < 8 / kPer; ++c) {
      const piece_t v = reinterpret_cast<const piece_t*>(p)[c];
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[c * kPer + j] = v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[j < live ? j * stride : 0];   // past them the first again
  }
  bf16x8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(j < live ? static_cast<float>(x[j]) : 0.f);
  return o;
}
template <typename T>
__device__ __forceinline__ void prepare_slot(const Prepare& q, int64_t i, int slot, int64_t place, const Pool& pool) {
  const int64_t rows = q.rows, cols = q.cols;
  const int R = pool.rank, r = slot_rank(pool, slot), rp = pool.rp, groups = rp / 8;
  const T* B = static_cast<const T*>(pool.B) + slot * (rows * R);
  const T* A = static_cast<const T*>(pool.A) + slot * (R * cols);
  const bf16x8 zero = {};
  if (q.Bp != nullptr) {
    if (i < rows * groups) {
      const int64_t row = i / groups;
      const int e = static_cast<int>(i % groups) * 8;
      *reinterpret_cast<bf16x8*>(q.Bp + (place * rows + row) * rp + e) = e < r ? pool_eight(B + row * R + e, 1, r - e) : zero;
      return;
    }
    i -= rows * groups;
  }
  if (q.Bt != nullptr) {   // neighbouring threads take neighbouring ranks, whose reads are one run
    if (i < q.rows8 / 8 * rp) {
      const int e = static_cast<int>(i % rp);
      const int64_t row = i / rp * 8;
      *reinterpret_cast<bf16x8*>(q.Bt + (place * rp + e) * q.rows8 + row) =
          e < r ? pool_eight(B + row * R + e, R, static_cast<int>(rows - row)) : zero;
      return;
    }
    i -= q.rows8 / 8 * rp;
  }
  if (q.Ab != nullptr) {
    if (i < cols / 8 * rp) {
      const int64_t e = i / (cols / 8), c = i % (cols / 8) * 8;
      *reinterpret_cast<bf16x8*>(q.Ab + (place * rp + e) * cols + c) = e < r ? pool_eight(A + e * cols + c, 1, 8) : zero;
      return;
    }
    i -= cols / 8 * rp;
  }
  if (q.At != nullptr && i < cols * groups) {   // neighbouring threads take neighbouring columns
    const int64_t c = i % cols;
    const int e = static_cast<int>(i / cols) * 8;
    *reinterpret_cast<bf16x8*>(q.At + (place * cols + c) * rp + e) = e < r ? pool_eight(A + e * cols + c, cols, r - e) : zero;
  }
}
__device__ __forceinline__ void zero_slot(float* out, int64_t n, int64_t i, int64_t threads) {
  for (; i < n; i += threads) out[i] = 0.f;
}
__device__ __forceinline__ void prepare_job(const Prepare& q, uint32_t wg, int threads, const PlanView& plan, const Pool& pool) {
  const int slot = wg / q.wgs;
  const int4 info = *reinterpret_cast<const int4*>(plan.info);
  if (info.z != plan.n || info.w != plan.slots) return;
  const int64_t i = static_cast<int64_t>(wg % q.wgs) * threads + threadIdx.x;
  if (plan.slot_used[slot + 1] == plan.slot_used[slot]) {
    if (q.dB != nullptr) zero_slot(q.dB + slot * (q.rows * pool.rank), q.rows * pool.rank, i, static_cast<int64_t>(q.wgs) * threads);
    if (q.dB != nullptr) zero_slot(q.dA + slot * (q.cols * pool.rank), q.cols * pool.rank, i, static_cast<int64_t>(q.wgs) * threads);
    return;
  }
  const int64_t place = used_place(plan, slot);
  if (pool.dt == LOFTQ_BF16) prepare_slot<__bf16>(q, i, slot, place, pool);
  else prepare_slot<float>(q, i, slot, place, pool);
}
__global__ __launch_bounds__(kThreads) void prepare_kernel(Prepare q, PlanView plan, Pool pool) {
  prepare_job(q, blockIdx.x, kThreads, plan, pool);
}

// ---- thin product over the features: a K range's part of keep(L) F^T ----
// A workgroup takes a tile and one range, whose steps of 64 its eight waves take in turn.  A wave multiplies
// all of the tile's tokens, so that a row of F serves 64 of them.  Its loads are whole 128-byte lines
// (eight lanes a row; in the order of the matrix cores' operands neighbouring lanes would read
// neighbouring rows, and a load would take the address unit three times as long), which pass through
// the wave's share of LDS into operands while the next step's are in flight: 16-byte piece c of row i
// lies at place c ^ (i / 2 % 8), so that any 16 rows read at one k meet every bank once.  The waves' sums
// meet in LDS.
//
// 8192 tokens of 11008 columns under a mask, rank 16: 49 us (3.7 TB/s), where the mask's 64-bit products, a word for
// four elements, cost about as much as the loads; 2048 of 4096 columns at rank 64 in fp32 factors: 16 us.
constexpr int kDownStep = 64;

template <int NT, int MT, typename F, bool kWide>
__device__ __forceinline__ void down_job(const AdapterDown& jb, int tile, int q, const TileInfo& t, const PlanView& plan,
                                         const Pool& pool, char* lds) {
  constexpr int XL = 2 * MT, FL = NT * static_cast<int>(sizeof(F)), kRowLanes = sizeof(F) == 2 ? 8 : 16;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), li = lane & 15, lg = lane >> 4;
  const int64_t K = jb.K, place = static_cast<int64_t>(tile) * kTile;
  const int width = static_cast<int>(K), steps = (width + kDownStep - 1) / kDownStep, per = (steps + jb.ks - 1) / jb.ks;
  const int begin = q * per, end = begin + per < steps ? begin + per : steps;
  const int r = slot_rank(pool, t.slot);
  const uint32_t thr = jb.drop.thr;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  const char* base = static_cast<const char*>(jb.F) + (jb.prepared ? used_place(plan, t.slot) : t.slot) * jb.slot_elems * sizeof(F);
  const int l_records = records_of(static_cast<int64_t>(plan.n) * K * 2), f_records = records_of(r * K * static_cast<int>(sizeof(F)));
  // load i: row 8 i + lane / 8 of the tile, piece lane % 8 of its 128 bytes
  int64_t row[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) row[i] = token_at(plan, place + 8 * i + lane / 8) * K + 8 * (lane % 8);
  uint64_t word[MT];   // of the mask: the generator's state for this lane's operands' first element
#pragma unroll
  for (int m = 0; m < MT; ++m)
    word[m] = thr != 0 ? key + ((static_cast<uint64_t>(token_at(plan, place + 16 * m + li) * K + 8 * lg) >> 2) + 1) * kMixGamma : 0;
  char* xs = lds + w * ((MT + NT) * 2048);
  char* fs = xs + MT * 2048;
  u32x4 x[XL], f[FL];
  auto load = [&](int step) __attribute__((always_inline)) {
    const int k0 = step * kDownStep;
    const bool any = step < end, live = k0 + 8 * (lane % 8) < width, flive = k0 + (kDownStep / kRowLanes) * (lane % kRowLanes) < width;
    const __amdgpu_buffer_rsrc_t xb = buffer_with(jb.L, any ? l_records : 0), fb = buffer_with(base, any ? f_records : 0);
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      if constexpr (kWide) {
        x[i] = u32x4{0u, 0u, 0u, 0u};
        if (any && live) x[i] = *reinterpret_cast<const u32x4*>(jb.L + row[i] + k0);
      } else {
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(xb, live ? static_cast<uint32_t>(row[i]) * 2 : kNowhere, k0 * 2, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      const uint32_t at = static_cast<uint32_t>((64 / kRowLanes * i + lane / kRowLanes) * width) * sizeof(F) + 16 * (lane % kRowLanes);
      f[i] = __builtin_amdgcn_raw_buffer_load_b128(fb, flive ? at : kNowhere, k0 * static_cast<int>(sizeof(F)), 0);
    }
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int p = 0; p < NT; ++p) acc[m][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  load(begin + w);
  for (int step = begin + w; step < end; step += kDownWaves) {
    const int at = (lane % 8 ^ (lane / 16 & 7)) << 4;   // row / 2 % 8 of row 8 i + lane / 8 is (4 i + lane / 16) % 8
#pragma unroll
    for (int i = 0; i < XL; ++i)
      *reinterpret_cast<u32x4*>(xs + (8 * i + lane / 8) * 128 + (at ^ ((4 * i & 7) << 4))) = x[i];
#pragma unroll
    for (int i = 0; i < FL; ++i) {
      if constexpr (sizeof(F) == 2) {
        *reinterpret_cast<u32x4*>(fs + (8 * i + lane / 8) * 128 + (at ^ ((4 * i & 7) << 4))) = f[i];
      } else {   // four ranks' rows a load, 16 lanes of four values each
        const int frow = 4 * i + lane / 16, piece = lane % 16 / 2;
        bf16x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = static_cast<__bf16>(__uint_as_float(f[i][j]));
        *reinterpret_cast<bf16x4*>(fs + frow * 128 + ((piece ^ (frow >> 1 & 7)) << 4) + (lane & 1) * 8) = o;
      }
    }
    __builtin_amdgcn_wave_barrier();   // a wave's own share: its reads come after its writes
    load(step + kDownWaves);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < kDownStep / 32; ++h) {
      u32x4 b[NT];
#pragma unroll
      for (int p = 0; p < NT; ++p) b[p] = *reinterpret_cast<const u32x4*>(fs + (16 * p + li) * 128 + (((4 * h + lg) ^ (li >> 1 & 7)) << 4));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        u32x4 v = *reinterpret_cast<const u32x4*>(xs + (16 * m + li) * 128 + (((4 * h + lg) ^ (li >> 1 & 7)) << 4));
        if (thr != 0) {   // 16 words of the mask a step
          const uint64_t z = word[m] + static_cast<uint64_t>(2 * step + h) * (8 * kMixGamma);
          const uint64_t w0 = mix64(z), w1 = mix64(z + kMixGamma);
          v[0] = drop_pair(v[0], w0, 0, thr);
          v[1] = drop_pair(v[1], w0, 2, thr);
          v[2] = drop_pair(v[2], w1, 0, thr);
          v[3] = drop_pair(v[3], w1, 2, thr);
        }
#pragma unroll
        for (int p = 0; p < NT; ++p) acc[m][p] = mfma16(v, b[p], acc[m][p]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  // the upper half of the waves parks its sums and the lower half adds them, until one is left
  float* part = reinterpret_cast<float*>(lds);
  auto at = [&](int wave, int m, int p, int v) { return (((wave * MT + m) * NT + p) * 4 + v) * 64 + lane; };
  __syncthreads();
#pragma unroll
  for (int left = kDownWaves / 2; left >= 1; left /= 2) {
    if (w >= left && w < 2 * left)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int p = 0; p < NT; ++p)
#pragma unroll
          for (int v = 0; v < 4; ++v) part[at(w - left, m, p, v)] = acc[m][p][v];
    __syncthreads();
    if (w < left)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int p = 0; p < NT; ++p)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][p][v] += part[at(w, m, p, v)];
    __syncthreads();
  }
  if (w > 0) return;
  float* out = jb.out + (static_cast<int64_t>(q) * plan.max_tiles * kTile + place) * (16 * NT);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int p = 0; p < NT; ++p)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int tok = 16 * m + 4 * lg + v;
        if (tok < t.count) out[tok * (16 * NT) + 16 * p + li] = acc[m][p][v];
      }
}

template <int NT, typename F, bool kWide>
__global__ __launch_bounds__(kDownThreads) void down_kernel(AdapterDownJobs jobs, Prepare prepare, PlanView plan, Pool pool) {
  // the waves' steps; four waves' sums, 4 NT KiB each, take no more
  __shared__ __align__(16) char lds[kDownWaves * (4 + NT) * 2048];
  uint32_t wg = blockIdx.x;
  const int which = wg < jobs.job[0].wgs ? 0 : 1;
  if (which == 1) wg -= jobs.job[0].wgs;
  const AdapterDown& jb = jobs.job[which];
  if (wg >= jb.wgs) {
    prepare_job(prepare, wg - jb.wgs, kDownThreads, plan, pool);
    return;
  }
  const int q = wg % jb.ks, tile = wg / jb.ks;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot < 0 || t.count == 0) return;
  if (t.count <= 16) down_job<NT, 1, F, kWide>(jb, tile, q, t, plan, pool, lds);
  else down_job<NT, 4, F, kWide>(jb, tile, q, t, plan, pool, lds);
}

// ---- the sum of the partials, and its pieces rank-major ----
__global__ __launch_bounds__(kThreads) void sum_kernel(AdapterSumJobs jobs, Prepare prepare, unsigned sums, PlanView plan, Pool pool) {
  __shared__ __align__(4) __bf16 turned[3 * 16][32 + 2];
  const int rp = pool.rp;
  if (blockIdx.x >= sums) {
    if (blockIdx.y == 0) prepare_job(prepare, blockIdx.x - sums, kThreads, plan, pool);
    return;
  }
  const AdapterSum& jb = jobs.job[blockIdx.y];
  if (jb.partials == nullptr) return;
  const int parts = rp / 16, p0 = static_cast<int>(blockIdx.x % parts) * 16;
  const int half = blockIdx.x / parts % 2, tile = blockIdx.x / parts / 2;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot < 0) return;
  const int64_t places = static_cast<int64_t>(plan.max_tiles) * kTile, place = static_cast<int64_t>(tile) * kTile + half * 32;
  const int r = slot_rank(pool, t.slot);
#pragma unroll
  for (int i = threadIdx.x; i < 32 * 16; i += kThreads) {
    const int tok = i / 16, p = p0 + i % 16;
    float x = 0.f;   // past the slot's own rank too, where the partials may hold an infinite row's products with zeros
    if (half * 32 + tok < t.count && p < r) {
      const float* src = jb.partials + (place + tok) * rp + p;
      int q = 0;
      for (; q + 4 <= jb.ks; q += 4) {   // four loads in flight, added in order
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = src[(q + e) * places * rp];
#pragma unroll
        for (int e = 0; e < 4; ++e) x += v[e];
      }
      for (; q < jb.ks; ++q) x += src[q * places * rp];
    }
    if (jb.sum != nullptr) jb.sum[(place + tok) * rp + p] = x;
    if (jb.St != nullptr) {
      __bf16 h[3];
      split3(x, h);
#pragma unroll
      for (int q = 0; q < 3; ++q) turned[q * 16 + i % 16][tok] = h[q];
    }
  }
  if (jb.St == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * 16 * 16; i += kThreads) {   // two tokens a store
    const int row = i / 16, tok = (i % 16) * 2;
    *reinterpret_cast<uint32_t*>(jb.St + (row / 16 * rp + p0 + row % 16) * places + place + tok) =
        *reinterpret_cast<const uint32_t*>(&turned[row][tok]);
  }
}

// ---- thin product over the ranks, with the addition ----
// A workgroup takes a tile and a run of blocks of 64 features, which its four waves share.  The partial
// sums of H are added while they are staged in LDS in three bf16 pieces.  The factor is the first
// operand, so a lane receives four consecutive features of a token.
//
// Bound by Y0 and Y: 8192 x 11008 in fp32 (dX, rank 16, masked) 129 us (5.6 TB/s), 8192 x 4096 in bf16 32 us (4.2 TB/s),
// 2048 x 11008 in fp32 at rank 64 47 us (3.8 TB/s: 45 KB of LDS let three workgroups share a CU, and the last round of
// workgroups fills half of them).
template <int KR, int G>
__device__ __forceinline__ void stage_pieces(const AdapterUp& u, const PlanView& plan, int64_t place, int count, int r, int rp,
                                             __bf16 (*hs)[kTile][32 * KR + 8]) {
  const int64_t places = static_cast<int64_t>(plan.max_tiles) * kTile;
#pragma unroll
  for (int i = threadIdx.x; i < 16 * G * 8 * KR; i += kThreads) {   // four ranks of a token
    const int tok = i / (8 * KR), p = i % (8 * KR) * 4;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (tok < count && p < r) {   // the partials hold whole 16s of ranks
      const float* src = u.H + (place + tok) * rp + p;
      int q = 0;
      for (; q + 4 <= u.ks; q += 4) {   // four loads in flight, added in order
        f32x4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const f32x4*>(src + (q + e) * places * rp);
#pragma unroll
        for (int e = 0; e < 4; ++e) x += v[e];
      }
      for (; q < u.ks; ++q) x += *reinterpret_cast<const f32x4*>(src + q * places * rp);
    }
    bf16x4 h[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p + j >= r) x[j] = 0.f;   // an infinite row's products with the zeros past the slot's rank are NaN
      __bf16 piece[3];
      split3(x[j], piece);
#pragma unroll
      for (int q = 0; q < 3; ++q) h[q][j] = piece[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<bf16x4*>(&hs[q][tok][p]) = h[q];
  }
}

// For outputs in whole 16-byte pieces and of less than 2^31 bytes: every load and store of the loop goes
// through buffer resources, without a branch.  A wave turns a group of 16 tokens' sums round in LDS, so that
// Y0 is loaded and Y stored in whole lines of a token (64-byte pieces of 16 tokens, as the matrix
// cores give them, cost a third of the rate); a group's registers take the next block's loads as soon
// as it is stored, so that four groups' loads are in flight all the time.
constexpr int kTurnLd = 64 + 4;   // 16 tokens written at one feature, or one read along its features, meet every bank once

template <typename O, int KR, int G, bool kMask>
__device__ __forceinline__ void up_blocks(const AdapterUp& u, const PlanView& plan, const Pool& pool, const TileInfo& t,
                                          int64_t place, int begin, int end, __bf16 (*hs)[kTile][32 * KR + 8],
                                          float (*turn)[kTurnLd]) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(O)), kLanes = 64 / kPer, kRows = 64 / kLanes, kPieces = 16 / kRows;
  typedef O piece_t __attribute__((ext_vector_type(kPer)));
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), li = lane & 15, lg = lane >> 4;
  const uint32_t N = static_cast<uint32_t>(u.features);
  const bool adapter = t.slot >= 0;
  const int slot = adapter ? t.slot : 0;   // without an adapter no rank of it is used
  const int r = adapter ? slot_rank(pool, slot) : 0;
  const int64_t ld = u.ld;
  const int all = records_of(static_cast<int64_t>(plan.n) * N * sizeof(O)), factor_records = records_of(N * ld * 2);
  const __bf16* factor = u.F + (u.prepared ? used_place(plan, slot) : slot) * (N * ld);
  const float g = pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f);
  const uint64_t key = kMask ? drop_key(u.drop) : 0;
  const __amdgpu_buffer_rsrc_t to = buffer_with(u.out, all);
  // piece c of group m: token 16 m + kRows c + lane / kLanes, features kPer (lane % kLanes) .. of a block
  const uint32_t n_lane = kPer * (lane % kLanes);
  uint32_t offset[G][kPieces];
#pragma unroll
  for (int m = 0; m < G; ++m)
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int tok = 16 * m + kRows * c + lane / kLanes;
      const uint32_t e = static_cast<uint32_t>(token_at(plan, place + tok)) * N + n_lane;
      offset[m][c] = tok < t.count ? e * static_cast<uint32_t>(sizeof(O)) : kNowhere;
    }
  u32x4 y[G][kPieces], f[4][KR];
  auto load_y = [&](int m, int block) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t from = buffer_with(u.in, u.in != nullptr && block < end ? all : 0);
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
      y[m][c] = __builtin_amdgcn_raw_buffer_load_b128(from, block * 64u + n_lane < N ? offset[m][c] : kNowhere,
                                                      block * 64 * static_cast<int>(sizeof(O)), 0);
  };
  auto load_factor = [&](int block) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t from = buffer_with(factor, block < end ? factor_records : 0);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int k = 0; k < KR; ++k) {
        const uint32_t n = static_cast<uint32_t>(block * 64 + 16 * a + li), p = 32 * k + 8 * lg;
        f[a][k] = __builtin_amdgcn_raw_buffer_load_b128(
            from, n < N && static_cast<int>(p) < r ? (n * static_cast<uint32_t>(ld) + p) * 2 : kNowhere, 0, 0);
      }
  };
  int block = begin + w;
#pragma unroll
  for (int m = 0; m < G; ++m) {
    load_y(m, block);
    __builtin_amdgcn_sched_barrier(0);   // in the order in which they are waited for
  }
  load_factor(block);
  stage_pieces<KR, G>(u, plan, place, t.count, r, pool.rp, hs);
  __syncthreads();
  for (; block < end; block += 4) {
    if (r % 8 != 0)   // ranks past the slot's own
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int k = 0; k < KR; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int p = 32 * k + 8 * lg + 2 * j;
            f[a][k][j] = p + 1 < r ? f[a][k][j] : (p < r ? f[a][k][j] & 0xFFFFu : 0u);
          }
#pragma unroll
    for (int m = 0; m < G; ++m) {
      f32x4 acc[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) acc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 2; q >= 0; --q)
#pragma unroll
        for (int k = 0; k < KR; ++k) {
          const u32x4 h = *reinterpret_cast<const u32x4*>(&hs[q][16 * m + li][32 * k + 8 * lg]);
#pragma unroll
          for (int a = 0; a < 4; ++a) acc[a] = mfma16(f[a][k], h, acc[a]);
        }
#pragma unroll
      for (int a = 0; a < 4; ++a) *reinterpret_cast<f32x4*>(&turn[li][16 * a + 4 * lg]) = acc[a];
      if (m == G - 1) load_factor(block + 4);
      __builtin_amdgcn_wave_barrier();   // a wave's own rows: its reads come after its writes
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        const piece_t before = __builtin_bit_cast(piece_t, y[m][c]);
        piece_t v;
#pragma unroll
        for (int e = 0; e < kPer / 4; ++e) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(&turn[kRows * c + lane / kLanes][n_lane + 4 * e]);
          const uint64_t bits =
              kMask ? drop_word(key, (offset[m][c] / static_cast<uint32_t>(sizeof(O)) + static_cast<uint32_t>(block * 64 + 4 * e)) >> 2) : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float old = static_cast<float>(before[4 * e + i]);
            const bool add = adapter && (!kMask || drop_keeps(bits, i, u.drop.thr));
            v[4 * e + i] = static_cast<O>(add ? fmaf(g, x[i], old) : old);
          }
        }
        // The block's offset is in the lanes' address and not in a scalar: behind a 16-byte store with a scalar offset the
        // compiler leaves no wait before the next write of the data's registers, and that write has been stored instead.
        const uint32_t at = offset[m][c] + static_cast<uint32_t>(block * 64) * static_cast<uint32_t>(sizeof(O));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), to, block * 64u + n_lane < N ? at : kNowhere, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
      load_y(m, block + 4);
      __builtin_amdgcn_sched_barrier(0);   // a group's operands and results do not take the next one's registers
    }
  }
}

template <typename O, int KR, bool kMask>
__global__ __launch_bounds__(kThreads) void up_kernel(AdapterUp u, PlanView plan, Pool pool, unsigned parts, int span) {
  __shared__ __align__(16) __bf16 hs[3][kTile][32 * KR + 8];   // 16 rows read at one rank meet every bank once
  __shared__ __align__(16) float turn[kThreads / 64][16][kTurnLd];
  const int tile = blockIdx.x / parts, begin = static_cast<int>(blockIdx.x % parts) * span;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot == -2 || t.count == 0 || (t.slot == -1 && u.in == u.out)) return;
  const int blocks = static_cast<int>((u.features + 63) / 64), end = begin + span < blocks ? begin + span : blocks;
  const int64_t place = static_cast<int64_t>(tile) * kTile;
  if (t.count <= 16) up_blocks<O, KR, 1, kMask>(u, plan, pool, t, place, begin, end, hs, turn[threadIdx.x >> 6]);
  else up_blocks<O, KR, 4, kMask>(u, plan, pool, t, place, begin, end, hs, turn[threadIdx.x >> 6]);
}

// For every other shape: 64-bit addresses, element by element.
template <typename O, int KR>
__global__ __launch_bounds__(kThreads) void up_any_kernel(AdapterUp u, PlanView plan, Pool pool, unsigned parts, int span) {
  __shared__ __align__(16) __bf16 hs[3][kTile][32 * KR + 8];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, li = lane & 15, lg = lane >> 4;
  const int tile = blockIdx.x / parts, begin = static_cast<int>(blockIdx.x % parts) * span;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot == -2 || t.count == 0 || (t.slot == -1 && u.in == u.out)) return;
  const int64_t N = u.features, ld = u.ld, place = static_cast<int64_t>(tile) * kTile;
  const int blocks = static_cast<int>((N + 63) / 64), end = begin + span < blocks ? begin + span : blocks;
  const bool adapter = t.slot >= 0;
  const int slot = adapter ? t.slot : 0, r = adapter ? slot_rank(pool, slot) : 0;
  const __amdgpu_buffer_rsrc_t factor = buffer_of(u.F + (u.prepared ? used_place(plan, slot) : slot) * (N * ld), N * ld * 2);
  const float g = pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f);
  const uint64_t key = u.drop.thr != 0 ? drop_key(u.drop) : 0;
  const O* in = static_cast<const O*>(u.in);
  O* out = static_cast<O*>(u.out);
  stage_pieces<KR, 4>(u, plan, place, t.count, r, pool.rp, hs);
  __syncthreads();
  for (int block = begin + w; block < end; block += 4)
    for (int a = 0; a < 4; ++a) {
      const int64_t n0 = static_cast<int64_t>(block) * 64 + 16 * a;
      u32x4 f[KR];
#pragma unroll
      for (int k = 0; k < KR; ++k) {
        const int64_t n = n0 + li;
        const int p = 32 * k + 8 * lg;
        f[k] = __builtin_amdgcn_raw_buffer_load_b128(factor, n < N && p < r ? static_cast<uint32_t>(n * ld + p) * 2 : kNowhere, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[k][j] = p + 2 * j + 1 < r ? f[k][j] : (p + 2 * j < r ? f[k][j] & 0xFFFFu : 0u);
      }
      for (int m = 0; 16 * m < t.count; ++m) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
          for (int k = 0; k < KR; ++k) acc = mfma16(f[k], *reinterpret_cast<const u32x4*>(&hs[q][16 * m + li][32 * k + 8 * lg]), acc);
        const int64_t row = token_at(plan, place + 16 * m + li) * N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t n = n0 + 4 * lg + i;
          if (16 * m + li >= t.count || n >= N) continue;
          const float x = in != nullptr ? static_cast<float>(in[row + n]) : 0.f;
          const bool add = adapter && (u.drop.thr == 0 ||
                                       drop_keeps(drop_word(key, static_cast<uint64_t>(row + n) >> 2), (row + n) & 3, u.drop.thr));
          out[row + n] = static_cast<O>(add ? fmaf(g, acc[i], x) : x);
        }
      }
    }
}

// ---- thin product over the tokens: the factors' gradients ----
// out[i][p] = sum_t keep(L)[t][i] S[t][p].  The matrix cores want each operand's K (tokens) in
// one lane, and L's tokens are rows: lane L loads 8 tokens x 8 features (16 bytes of 8
// rows) and turns the 8 x 8 block round in its registers, which gives the operands of 8
// products, the j-th for features 8 (L%16) + j.  A workgroup takes 128 features and a chunk of
// one slot's tiles, which its four waves share 32 tokens at a time; past 32 ranks two waves share
// a step, half of the ranks each.  kRankMajor (dA): S is the first operand, so a lane holds 8
// consecutive features of a rank; else (dB) a lane's rank is L%16.
//
// 8192 tokens of 4096 + 11008 features at rank 16, X masked: 62 us (4.0 TB/s); 2048 of 11008 + 4096 at rank 64: 38 us, bound
// by the loads' latency at two waves a SIMD (S's pieces a step ahead need more registers than there are: a fifth longer).
template <int NR, bool kRankMajor, bool kWide>
__device__ __forceinline__ void grad_job(const AdapterGrad& jb, uint32_t group_at, int at_chunk, const PlanView& plan, const Pool& pool,
                                         float (*part)[8 * (NR > 2 ? 2 : NR) * 4 * 64]) {
  constexpr int kParts = NR > 2 ? 2 : 1, NT = NR > 2 ? 2 : NR, kWaves = 4 / kParts;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave % kParts, w = wave / kParts, tile0 = half * NT;
  const int64_t F = jb.F, places = static_cast<int64_t>(plan.max_tiles) * kTile;
  const int64_t group = group_at;
  const int4 info = *reinterpret_cast<const int4*>(plan.info);
  if (info.z != plan.n || info.w != plan.slots || at_chunk >= info.y) return;
  const int4 chunk = plan.chunks[at_chunk];
  const int slot = chunk.x, first = chunk.y, tiles = chunk.z;
  if (static_cast<unsigned>(slot) >= static_cast<unsigned>(plan.slots) || first < 0 || tiles < 1 || first + tiles > plan.max_tiles)
    return;
  const bool whole = chunk.w == 1;   // the slot's only one
  if (!whole && at_chunk >= plan.max_parts) return;
  const int64_t f0 = group * 128 + 8 * li, f = f0 < F ? f0 : F - 8;   // 8 | F
  const int steps = 2 * tiles - (tile_info(plan, first + tiles - 1).count > 32 ? 0 : 1);
  const uint32_t thr = kRankMajor ? jb.drop.thr : 0;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  f32x4 acc[8][NT];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t place0 = static_cast<int64_t>(first) * kTile;
  u32x4 x[2][8], b[3][NT];
  uint32_t token[2][8];
  const uint32_t width = static_cast<uint32_t>(F), bat = static_cast<uint32_t>(li * places + 8 * lg) * 2;
  const int l_records = records_of(static_cast<int64_t>(plan.n) * F * 2);
  int4 lo, hi;   // the next step's tokens, loaded a step before they are wanted
  auto load_rows = [&](int s) __attribute__((always_inline)) {
    const int32_t* rows = plan.rows + place0 + 32 * static_cast<int64_t>(s < steps ? s : steps - 1) + 8 * lg;
    lo = *reinterpret_cast<const int4*>(rows);
    hi = *reinterpret_cast<const int4*>(rows + 4);
  };
  auto load = [&](int set, int s) __attribute__((always_inline)) {
    const int t[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) token[set][i] = static_cast<unsigned>(t[i]) < static_cast<unsigned>(plan.n) ? t[i] : 0;
    const __amdgpu_buffer_rsrc_t xb = buffer_with(jb.L, s < steps ? l_records : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (kWide)
        x[set][i] = *reinterpret_cast<const u32x4*>(jb.L + token[set][i] * F + f);
      else
        x[set][i] = __builtin_amdgcn_raw_buffer_load_b128(xb, (token[set][i] * width + static_cast<uint32_t>(f)) * 2, 0, 0);
    }
    load_rows(s + kWaves);
  };
  auto load_s = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) {   // of an odd number of rank tiles the last half's second repeats the first
        const int tile = tile0 + t < NR ? tile0 + t : tile0;
        b[h][t] = __builtin_amdgcn_raw_buffer_load_b128(
            buffer_at(jb.St + static_cast<int64_t>(h * 16 * NR + tile * 16) * places + place0 + 32 * static_cast<int64_t>(s), s < steps), bat, 0, 0);
      }
  };
  auto multiply = [&](int set) __attribute__((always_inline)) {
    if (thr != 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[set][i] = drop8(x[set][i], key, static_cast<uint64_t>(token[set][i] * F + f), thr);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4 lo, hi;   // features 2 c and 2 c + 1: tokens 0 .. 7
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(x[set][2 * i + 1][c], x[set][2 * i][c], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(x[set][2 * i + 1][c], x[set][2 * i][c], 0x07060302u);
      }
#pragma unroll
      for (int h = 0; h < 3; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[2 * c][t] = kRankMajor ? mfma16(b[h][t], lo, acc[2 * c][t]) : mfma16(lo, b[h][t], acc[2 * c][t]);
          acc[2 * c + 1][t] = kRankMajor ? mfma16(b[h][t], hi, acc[2 * c + 1][t]) : mfma16(hi, b[h][t], acc[2 * c + 1][t]);
        }
    }
  };
  if (w < steps) {
    load_rows(w);
    load(0, w);
    for (int s = w; s < steps; s += 2 * kWaves) {
      load_s(s);
      load(1, s + kWaves);
      multiply(0);
      if (s + kWaves >= steps) break;
      load_s(s + kWaves);
      load(0, s + 2 * kWaves);
      multiply(1);
    }
  }
  // of four waves 2 and 3 park their sums, 0 and 1 add them; then 1 parks and 0 adds
  auto at = [&](int j, int t, int v) { return ((j * NT + t) * 4 + v) * 64 + lane; };
  auto park = [&](float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) to[at(j, t, v)] = acc[j][t][v];
  };
  auto add = [&](const float* from) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][t][v] += from[at(j, t, v)];
  };
  if constexpr (kWaves == 4) {
    if (w >= 2) park(part[w - 2]);
    __syncthreads();
    if (w < 2) add(part[w]);
    __syncthreads();
  }
  if (w == 1) park(part[half]);
  __syncthreads();
  if (w != 0) return;
  add(part[half]);
  // one chunk: the gradient itself; more: a partial sum with whole padded ranks and features
  const int64_t nf = whole ? jb.nf : F;
  const int nr = whole ? pool.rank : 16 * NR;
  const float coef = whole ? pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f) : 1.f;
  const int r = slot_rank(pool, slot);   // past it zeros, where an infinity of L has met them too
  float* o = whole ? jb.out + slot * (nf * nr) : jb.partials + at_chunk * (F * 16 * NR);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (tile0 + t) * 16 + (kRankMajor ? 4 * lg + v : li) < r ? coef * acc[j][t][v] : 0.f;
      if constexpr (kRankMajor) {
        const int p = (tile0 + t) * 16 + 4 * lg + v;   // features f0 .. f0 + 7
        if (p < nr && f0 < F)                          // nf == F here, and 8 | F
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<f32x4*>(o + p * nf + f0 + 4 * h) = f32x4{y[4 * h], y[4 * h + 1], y[4 * h + 2], y[4 * h + 3]};
      } else {
        const int p = (tile0 + t) * 16 + li;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t i = group * 128 + 8 * (4 * lg + v) + j;
          if (i < nf && p < nr) o[i * nr + p] = y[j];
        }
      }
    }
}

// job 0: dB over dY, `first` groups of features; job 1: dA over X, `second` groups.  Both jobs of a chunk before the next
// chunk, so that the workgroups of chunks that the batch does not have come last and the others spread over the CUs.
template <int NT, bool kWide>
__global__ __launch_bounds__(kThreads, 2) void grad_kernel(AdapterGradJobs jobs, PlanView plan, Pool pool, uint32_t first,
                                                           uint32_t second) {
  __shared__ float part[2][8 * (NT > 2 ? 2 : NT) * 4 * 64];
  const uint32_t chunk = blockIdx.x / (first + second), group = blockIdx.x % (first + second);
  if (group < first)
    grad_job<NT, false, kWide>(jobs.job[0], group, static_cast<int>(chunk), plan, pool, part);
  else
    grad_job<NT, true, kWide>(jobs.job[1], group - first, static_cast<int>(chunk), plan, pool, part);
}

// gain times the sum of the partials of a slot with several chunks, in their order; zeros for a batch without tokens
__global__ __launch_bounds__(kThreads) void grad_sum_kernel(AdapterGradJobs jobs, PlanView plan, Pool pool, uint32_t first) {
  const bool rank_major = blockIdx.x >= first;
  const AdapterGrad& jb = jobs.job[rank_major ? 1 : 0];
  const int slot = blockIdx.y, R = pool.rank, rp = pool.rp;
  int chunk = 0, chunks = 0;
  if (plan.n > 0) {
    const int4 info = *reinterpret_cast<const int4*>(plan.info);
    if (info.z != plan.n || info.w != plan.slots) return;
    chunk = plan.slot_parts[slot];
    chunks = plan.slot_parts[slot + 1] - chunk;
    if (chunks < 2 || chunk < 0 || chunk + chunks > plan.max_parts) return;
  }
  const int64_t i = (static_cast<int64_t>(blockIdx.x - (rank_major ? first : 0)) * kThreads + threadIdx.x) * 4, nf = jb.nf, all = nf * R;
  if (i >= all) return;
  const float g = pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f);
  float* out = jb.out + slot * all + i;
  const float* src = jb.partials + chunk * (jb.F * rp);
  if (all % 4 == 0 && (rank_major || R % 4 == 0)) {   // four elements in a row in either form
    const uint32_t e = static_cast<uint32_t>(i), per = static_cast<uint32_t>(R);
    const int64_t at = rank_major ? i : static_cast<int64_t>(e / per) * rp + e % per;   // nf == F for dA
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < chunks; ++q) x += *reinterpret_cast<const f32x4*>(src + q * (jb.F * rp) + at);
    if (chunks > 0) x *= g;
    *reinterpret_cast<f32x4*>(out) = x;
    return;
  }
  for (int j = 0; j < 4 && i + j < all; ++j) {
    const int64_t at = rank_major ? i + j : (i + j) / R * rp + (i + j) % R;
    float x = 0.f;
    for (int q = 0; q < chunks; ++q) x += src[q * (jb.F * rp) + at];
    out[j] = chunks > 0 ? g * x : 0.f;
  }
}

__global__ __launch_bounds__(kThreads) void pad_kernel(const __bf16* __restrict__ in, __bf16* __restrict__ out, int64_t n,
                                                       int64_t from, int64_t to) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, per_row = to / 8;
  const int64_t row = id / per_row, c = id % per_row * 8;
  if (row >= n) return;
  bf16x8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = c + j < from ? in[row * from + c + j] : static_cast<__bf16>(0.f);
  *reinterpret_cast<bf16x8*>(out + row * to + c) = o;
}

unsigned blocks_for(int64_t threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

// K ranges for about `tiles` tiles: workgroups for every CU several times over (8192 tokens of 11008 columns at rank 16:
// 62 us with 133 workgroups in all, 50 with 399, 47 with 931, 53 with 1995), fewer of them where the waves' sums are larger
// (2048 tokens of 11008 + 4096 columns at rank 64: 57 us with 74, 34 with 148, 32 with 518, 36 with 814); each range has a
// step for every wave
int splits_for(int64_t tiles, int64_t K, int rp) {
  int64_t ks = 1024 / (rp / 16) / tiles;
  const int64_t most = (K + kDownStep - 1) / kDownStep / kDownWaves;
  if (ks > most) ks = most;
  return static_cast<int>(ks < 1 ? 1 : (ks > 16 ? 16 : ks));
}
// how many tiles a batch may have, the slots' last ones half of the time
int64_t tiles_of(int64_t n, int slots) { return 1 + n / kTile + (n < slots ? n : slots) / 2; }

}  // namespace

#define LQ_BY_RANK(rp, CALL) \
  switch ((rp) / 16) {       \
    case 1: CALL(1); break;  \
    case 2: CALL(2); break;  \
    case 3: CALL(3); break;  \
    default: CALL(4); break; \
  }

int adapters_down_splits(int64_t n, int slots, int64_t K, int rp) { return splits_for(tiles_of(n, slots), K, rp); }

// A batch has at most twice tiles_of() tiles, so that its ranges and tiles are at most twice what splits_for() divides.
int64_t adapters_down_floats_bound(int64_t n, int slots, int64_t K, int rp) {
  const int64_t tiles = plan_layout(n, slots).max_tiles, most = tiles * splits_for(1, K, 16), divided = 2 * 1024 / (rp / 16);
  const int64_t bound = most < divided ? most : divided;
  return (bound > tiles ? bound : tiles) * kTile * rp;
}

static unsigned prepare_wgs(const Prepare& q, const Pool& pool, int threads) {
  const int64_t rp = pool.rp, work = (q.Bp ? q.rows * (rp / 8) : 0) + (q.Bt ? q.rows8 / 8 * rp : 0) +
                                     (q.Ab ? q.cols / 8 * rp : 0) + (q.At ? q.cols * (rp / 8) : 0);
  return static_cast<unsigned>((work + threads - 1) / threads);
}

hipError_t launch_adapters_prepare(Prepare q, const PlanView& plan, const Pool& pool, hipStream_t s) {
  q.wgs = prepare_wgs(q, pool, kThreads);
  if (q.wgs == 0) return hipSuccess;
  LQ_LAUNCH("adapters_prepare", prepare_kernel, dim3(q.wgs * pool.slots), dim3(kThreads), 0, s, q, plan, pool);
  return hipGetLastError();
}

hipError_t launch_adapters_down(AdapterDownJobs jobs, loftq_dtype_t factor, const Prepare& prepare, const PlanView& plan,
                                const Pool& pool, hipStream_t s) {
  Prepare q = prepare;
  q.wgs = prepare_wgs(q, pool, kDownThreads);
  bool wide = false;   // 32-bit offsets reach the tokens' rows
  for (AdapterDown& j : jobs.job) {
    j.wgs = j.L != nullptr ? static_cast<unsigned>(plan.max_tiles * j.ks) : 0;
    wide = wide || (j.L != nullptr && plan.n * j.K * 2 >= (int64_t(1) << 31));
  }
  const dim3 grid(jobs.job[0].wgs + jobs.job[1].wgs + q.wgs * pool.slots), block(kDownThreads);
#define LQ_DOWN_KERNEL(NT, F, W) LQ_LAUNCH("adapters_down", (down_kernel<NT, F, W>), grid, block, 0, s, jobs, q, plan, pool)
#define LQ_DOWN(NT)                                                \
  do {                                                             \
    if (factor == LOFTQ_BF16 && wide) LQ_DOWN_KERNEL(NT, __bf16, true); \
    else if (factor == LOFTQ_BF16) LQ_DOWN_KERNEL(NT, __bf16, false);   \
    else if (wide) LQ_DOWN_KERNEL(NT, float, true);                \
    else LQ_DOWN_KERNEL(NT, float, false);                         \
  } while (0)
  LQ_BY_RANK(pool.rp, LQ_DOWN)
#undef LQ_DOWN
#undef LQ_DOWN_KERNEL
  return hipGetLastError();
}

hipError_t launch_adapters_sum(AdapterSumJobs jobs, const Prepare& prepare, const PlanView& plan, const Pool& pool, hipStream_t s) {
  Prepare q = prepare;
  q.wgs = prepare_wgs(q, pool, kThreads);
  const unsigned sums = static_cast<unsigned>(2 * plan.max_tiles * (pool.rp / 16));
  LQ_LAUNCH("adapters_sum", sum_kernel, dim3(sums + q.wgs * pool.slots, jobs.job[1].partials != nullptr ? 2 : 1), dim3(kThreads), 0, s,
            jobs, q, sums, plan, pool);
  return hipGetLastError();
}

hipError_t launch_adapters_up(const AdapterUp& u, const PlanView& plan, const Pool& pool, hipStream_t s) {
  const int64_t blocks = (u.features + 63) / 64, size = u.odt == LOFTQ_BF16 ? 2 : 4;
  // about 2048 workgroups; where 512 remain each wave has two blocks, so that one's loads pass over the other (2048 tokens
  // x 11008, rank 64: 50 us with one, 48 with two; 2048 x 4096 has too few: 20 and 21)
  const int64_t work = tiles_of(plan.n, plan.slots) * blocks, least = work / 8 >= 512 ? 8 : 4;
  int64_t span = work / 2048 / 4 * 4;
  span = span < least ? least : (span > 64 ? 64 : span);
  const unsigned parts = static_cast<unsigned>((blocks + span - 1) / span);
  const dim3 grid(static_cast<unsigned>(plan.max_tiles) * parts), block(kThreads);
  const bool whole = u.features % (16 / size) == 0 && plan.n * u.features * size < (int64_t(1) << 31), mask = u.drop.thr != 0;
#define LQ_UP_KERNEL(...) LQ_LAUNCH("adapters_up", (__VA_ARGS__), grid, block, 0, s, u, plan, pool, parts, static_cast<int>(span))
#define LQ_UP(O, KR)                                        \
  do {                                                      \
    if (!whole) LQ_UP_KERNEL(up_any_kernel<O, KR>);         \
    else if (mask) LQ_UP_KERNEL(up_kernel<O, KR, true>);    \
    else LQ_UP_KERNEL(up_kernel<O, KR, false>);             \
  } while (0)
  if (u.odt == LOFTQ_BF16) {
    if (pool.rp <= 32) LQ_UP(__bf16, 1);
    else LQ_UP(__bf16, 2);
  } else {
    if (pool.rp <= 32) LQ_UP(float, 1);
    else LQ_UP(float, 2);
  }
#undef LQ_UP
#undef LQ_UP_KERNEL
  return hipGetLastError();
}

hipError_t launch_adapters_grad(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s) {
  unsigned groups[2];
  for (int j = 0; j < 2; ++j) groups[j] = static_cast<unsigned>((jobs.job[j].F + 127) / 128);
  // 32-bit offsets reach the tokens' rows
  const bool wide = plan.n * jobs.job[0].F * 2 >= (int64_t(1) << 31) || plan.n * jobs.job[1].F * 2 >= (int64_t(1) << 31);
#define LQ_GRAD_KERNEL(NT, W) \
  LQ_LAUNCH("adapters_grad", (grad_kernel<NT, W>), dim3((groups[0] + groups[1]) * plan.max_chunks), dim3(kThreads), 0, s, jobs, plan, pool, \
            groups[0], groups[1])
#define LQ_GRAD(NT)                       \
  do {                                    \
    if (wide) LQ_GRAD_KERNEL(NT, true);   \
    else LQ_GRAD_KERNEL(NT, false);       \
  } while (0)
  LQ_BY_RANK(pool.rp, LQ_GRAD)
#undef LQ_GRAD
#undef LQ_GRAD_KERNEL
  return hipGetLastError();
}

hipError_t launch_adapters_grad_sum(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s) {
  const unsigned first = blocks_for((jobs.job[0].nf * pool.rank + 3) / 4), second = blocks_for((jobs.job[1].nf * pool.rank + 3) / 4);
  LQ_LAUNCH("adapters_grad_sum", grad_sum_kernel, dim3(first + second, pool.slots), dim3(kThreads), 0, s, jobs, plan, pool, first);
  return hipGetLastError();
}

hipError_t launch_adapters_pad(const __bf16* in, __bf16* out, int64_t n, int64_t from, int64_t to, hipStream_t s) {
  LQ_LAUNCH("adapters_pad", pad_kernel, dim3(blocks_for(n * (to / 8))), dim3(kThreads), 0, s, in, out, n, from, to);
  return hipGetLastError();
}

}  // namespace loftq
