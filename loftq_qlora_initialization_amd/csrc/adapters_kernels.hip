// Products of many adapters beside one shared weight: each token with the factors of its own slot.
//
// The plan has sorted the tokens into tiles of one slot each, so a tile's products are dense; its
// rows are gathered from X and scattered to Y by token number, whole rows at a time.  All of it
// is bound by loads and stores: X, Y0 and Y once each, a slot's factors once for every tile that
// shares a CU's or an XCD's cache.
//
// v_mfma_f32_16x16x32_bf16: lane L supplies A[L%16][8(L/16) + j] and
// B[8(L/16) + j][L%16] (j = 0..7) and receives D[4(L/16) + v][L%16] in element v.
#include "adapters.h"
#include "buffer.h"

namespace loftq {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kNowhere = 0x7FFFFFFFu;   // an offset past every resource: loads give zeros

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 8 values of a masked row, elements e .. e + 7 of the flattening (e % 8 == 0)
__device__ __forceinline__ u32x4 drop8(u32x4 v, uint64_t key, uint64_t e, uint32_t thr) {
  const uint64_t w0 = drop_word(key, e >> 2), w1 = drop_word(key, (e >> 2) + 1);
  v[0] = drop_pair(v[0], w0, 0, thr);
  v[1] = drop_pair(v[1], w0, 2, thr);
  v[2] = drop_pair(v[2], w1, 0, thr);
  v[3] = drop_pair(v[3], w1, 2, thr);
  return v;
}

// x = h0 + h1 + h2 in bf16, each the rounding of what the ones before leave (24 bits in all; an infinity
// or a NaN is all in the first)
__device__ __forceinline__ void split3(float x, __bf16 (&h)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    h[q] = static_cast<__bf16>(x);
    x = __builtin_isfinite(static_cast<float>(h[q])) ? x - static_cast<float>(h[q]) : 0.f;
  }
}

// A tile of a plan that belongs to this call's sizes; slot -1 has no adapter, -2 is no tile.
struct TileInfo {
  int slot, count;
};
__device__ __forceinline__ TileInfo tile_info(const PlanView& p, int tile) {
  const int4 info = *reinterpret_cast<const int4*>(p.info);
  const bool ours = info.z == p.n && info.w == p.slots;
  if (!ours || tile >= info.x) return TileInfo{-2, 0};
  const int4 t = p.tiles[tile];
  return TileInfo{t.x >= p.slots ? -2 : t.x, t.z < 0 ? 0 : (t.z > kTile ? kTile : t.z)};
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

// Eight elements of a factor for consecutive ranks or columns, as bf16.
template <typename F>
struct Factor;
template <>
struct Factor<__bf16> {
  static constexpr uint32_t kSize = 2;
  static __device__ __forceinline__ u32x4 run(__amdgpu_buffer_rsrc_t b, uint32_t at) {   // eight in a row
    return __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
  }
  static __device__ __forceinline__ u32x4 strided(__amdgpu_buffer_rsrc_t b, const uint32_t (&at)[8]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(b, at[2 * j], 0, 0)) |
             static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(b, at[2 * j + 1], 0, 0)) << 16;
    return v;
  }
};
template <>
struct Factor<float> {
  static constexpr uint32_t kSize = 4;
  static __device__ __forceinline__ u32x4 round8(const float (&x)[8]) {
    bf16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(x[j]);
    return __builtin_bit_cast(u32x4, o);
  }
  static __device__ __forceinline__ u32x4 run(__amdgpu_buffer_rsrc_t b, uint32_t at) {
    const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
    const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(b, at == kNowhere ? at : at + 16, 0, 0);
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(j < 4 ? lo[j & 3] : hi[j & 3]);
    return round8(x);
  }
  static __device__ __forceinline__ u32x4 strided(__amdgpu_buffer_rsrc_t b, const uint32_t (&at)[8]) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, at[j], 0, 0));
    return round8(x);
  }
};

// ---- thin product over the features: a K range's part of keep(L) F^T ----
// A workgroup takes half a tile (32 tokens) and one range, which its eight waves share U steps of
// 32 at a time.  All loads of U steps are issued before the first product.  The waves' sums meet
// in LDS.
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / 64;

template <int NT, typename F, bool kOverB>
__device__ __forceinline__ void down_job(const AdapterDown& jb, uint32_t wg, const PlanView& plan, const Pool& pool,
                                         float (*part)[2 * NT * 4 * 64]) {
  constexpr int U = NT <= 2 ? 4 : 2;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), li = lane & 15, lg = lane >> 4;
  const int q = wg % jb.ks, half = wg / jb.ks % 2, tile = wg / jb.ks / 2;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot < 0 || half * 32 >= t.count) return;
  const int64_t K = jb.K, place = static_cast<int64_t>(tile) * kTile + half * 32;
  const int steps = static_cast<int>((K + 31) / 32), per = (steps + jb.ks - 1) / jb.ks;
  const int begin = q * per, end = begin + per < steps ? begin + per : steps;
  const int r = slot_rank(pool, t.slot), R = pool.rank;
  const uint32_t thr = kOverB ? 0 : jb.drop.thr;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  const __bf16* row[2];
  uint64_t element[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int64_t token = token_at(plan, place + 16 * m + li);
    row[m] = jb.L + token * K;
    element[m] = static_cast<uint64_t>(token * K);
  }
  // A: rank p's row is K columns (records end with the slot's rank); B: column p of `rows` rows
  const int64_t slot_elems = kOverB ? jb.rows * R : static_cast<int64_t>(R) * K;
  const char* base = static_cast<const char*>(kOverB ? pool.B : pool.A) + t.slot * slot_elems * Factor<F>::kSize;
  const __amdgpu_buffer_rsrc_t rsrc = buffer_of(base, (kOverB ? slot_elems : r * K) * Factor<F>::kSize);
  f32x4 acc[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int p = 0; p < NT; ++p) acc[m][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = begin + w * U; s0 < end; s0 += kDownWaves * U) {
    u32x4 x[U][2], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s0 + u) * 32 + 8 * lg;
      const bool live = s0 + u < end && k < K;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        x[u][m] = u32x4{0u, 0u, 0u, 0u};
        if (live) x[u][m] = *reinterpret_cast<const u32x4*>(row[m] + k);
      }
#pragma unroll
      for (int p = 0; p < NT; ++p) {
        const int rank = 16 * p + li;
        if constexpr (kOverB) {
          uint32_t at[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) at[j] = live && rank < r ? static_cast<uint32_t>((k + j) * R + rank) * Factor<F>::kSize : kNowhere;
          b[u][p] = Factor<F>::strided(rsrc, at);
        } else {
          b[u][p] = Factor<F>::run(rsrc, live ? static_cast<uint32_t>(rank * K + k) * Factor<F>::kSize : kNowhere);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        u32x4 v = x[u][m];
        if (thr != 0) v = drop8(v, key, element[m] + static_cast<uint64_t>((s0 + u) * 32 + 8 * lg), thr);
#pragma unroll
        for (int p = 0; p < NT; ++p) acc[m][p] = mfma16(v, b[u][p], acc[m][p]);
      }
  }
  // the upper half of the waves parks its sums and the lower half adds them, until one is left
  auto at = [&](int m, int p, int v) { return ((m * NT + p) * 4 + v) * 64 + lane; };
#pragma unroll
  for (int left = kDownWaves / 2; left >= 1; left /= 2) {
    if (w >= left && w < 2 * left)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int p = 0; p < NT; ++p)
#pragma unroll
          for (int v = 0; v < 4; ++v) part[w - left][at(m, p, v)] = acc[m][p][v];
    __syncthreads();
    if (w < left)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int p = 0; p < NT; ++p)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][p][v] += part[w][at(m, p, v)];
    __syncthreads();
  }
  if (w > 0) return;
  float* out = jb.out + (static_cast<int64_t>(q) * plan.max_tiles * kTile + place) * (16 * NT);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int p = 0; p < NT; ++p)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int tok = 16 * m + 4 * lg + v;
        if (half * 32 + tok < t.count) out[tok * (16 * NT) + 16 * p + li] = acc[m][p][v];
      }
}

template <int NT, typename F>
__global__ __launch_bounds__(kDownThreads) void down_kernel(AdapterDownJobs jobs, PlanView plan, Pool pool) {
  __shared__ float part[kDownWaves / 2][2 * NT * 4 * 64];
  if (blockIdx.x < jobs.job[0].wgs)
    down_job<NT, F, true>(jobs.job[0], blockIdx.x, plan, pool, part);
  else
    down_job<NT, F, false>(jobs.job[1], blockIdx.x - jobs.job[0].wgs, plan, pool, part);
}

// ---- the sum of the partials, and its pieces rank-major ----
constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void sum_kernel(AdapterSumJobs jobs, PlanView plan, int rp) {
  __shared__ __align__(4) __bf16 turned[3 * 16][32 + 2];
  const AdapterSum& jb = jobs.job[blockIdx.y];
  if (jb.partials == nullptr) return;
  const int parts = rp / 16, p0 = static_cast<int>(blockIdx.x % parts) * 16;
  const int half = blockIdx.x / parts % 2, tile = blockIdx.x / parts / 2;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot < 0) return;
  const int64_t places = static_cast<int64_t>(plan.max_tiles) * kTile, place = static_cast<int64_t>(tile) * kTile + half * 32;
#pragma unroll
  for (int i = threadIdx.x; i < 32 * 16; i += kThreads) {
    const int tok = i / 16, p = p0 + i % 16;
    float x = 0.f;
    if (half * 32 + tok < t.count)
      for (int q = 0; q < jb.ks; ++q) x += jb.partials[(q * places + place + tok) * rp + p];
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
// A workgroup takes a tile and 256 features, 64 a wave.  The factor is the first operand; its rows
// are dealt to the four matrix tiles of a wave so that a lane receives 16 consecutive features of a
// token (tile a, element v of lane group g: feature 16 g + 4 a + v): whole lines of Y0 and Y a
// token.  The partial sums of H are added while they are staged in LDS in three bf16 pieces.
template <typename O, typename F, int KR, bool kVec, bool kOverA>
__global__ __launch_bounds__(kThreads) void up_kernel(AdapterUp u, PlanView plan, Pool pool, unsigned blocks) {
  constexpr int kLd = 32 * KR + 8;   // 16 bytes past whole 64: 16 rows read at one rank meet every bank once
  constexpr int kPer = 16 / static_cast<int>(sizeof(O)), kPieces = 16 / kPer;
  typedef O piece_t __attribute__((ext_vector_type(kPer)));
  __shared__ __align__(16) __bf16 hs[3][kTile][kLd];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, li = lane & 15, lg = lane >> 4;
  const int tile = blockIdx.x / blocks;
  const TileInfo t = tile_info(plan, tile);
  if (t.slot == -2 || (t.slot == -1 && u.in == u.out)) return;
  const int64_t N = u.features, n0 = static_cast<int64_t>(blockIdx.x % blocks) * 256 + w * 64, f0 = n0 + 16 * lg;
  const int64_t place = static_cast<int64_t>(tile) * kTile;
  const O* in = static_cast<const O*>(u.in);
  O* out = static_cast<O*>(u.out);

  f32x4 acc[4];   // of one 16-token group
  // y = in + g acc (acc where the mask keeps), or a copy of `in`
  auto store = [&](int m, bool adapter, float g, uint64_t key) __attribute__((always_inline)) {
    if (16 * m + li >= t.count) return;
    const int64_t at = token_at(plan, place + 16 * m + li) * N + f0;
    float y[16];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      if constexpr (kVec) {
        piece_t v = {};
        if (in != nullptr && f0 + c * kPer < N) v = *reinterpret_cast<const piece_t*>(in + at + c * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j) y[c * kPer + j] = static_cast<float>(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          y[c * kPer + j] = in != nullptr && f0 + c * kPer + j < N ? static_cast<float>(in[at + c * kPer + j]) : 0.f;
      }
    }
    if (adapter)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const uint64_t word = kOverA && u.drop.thr != 0 ? drop_word(key, static_cast<uint64_t>(at + 4 * a) >> 2) : ~0ull;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (!kOverA || drop_keeps(word, v, u.drop.thr)) y[4 * a + v] = fmaf(g, acc[a][v], y[4 * a + v]);
      }
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      if constexpr (kVec) {
        piece_t v;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = static_cast<O>(y[c * kPer + j]);
        if (f0 + c * kPer < N) *reinterpret_cast<piece_t*>(out + at + c * kPer) = v;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (f0 + c * kPer + j < N) out[at + c * kPer + j] = static_cast<O>(y[c * kPer + j]);
      }
    }
  };
  if (t.slot < 0) {
    for (int m = 0; 16 * m < t.count; ++m) store(m, false, 0.f, 0);
    return;
  }

  // the factor's operands: rank 32 k + 8 lg + j of feature n0 + 16 (li / 4) + 4 a + li % 4
  const int r = slot_rank(pool, t.slot), R = pool.rank;
  const char* base = static_cast<const char*>(kOverA ? pool.A : pool.B) + t.slot * (N * R) * Factor<F>::kSize;
  const __amdgpu_buffer_rsrc_t rsrc = buffer_of(base, N * R * Factor<F>::kSize);
  u32x4 f[4][KR];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int k = 0; k < KR; ++k) {
      const int64_t n = n0 + 16 * (li >> 2) + 4 * a + (li & 3);
      const int p = 32 * k + 8 * lg;
      if (!kOverA && R % 8 == 0 && r == R) {
        f[a][k] = Factor<F>::run(rsrc, n < N && p < R ? static_cast<uint32_t>(n * R + p) * Factor<F>::kSize : kNowhere);
      } else {
        uint32_t at[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          at[j] = n < N && p + j < r
                      ? static_cast<uint32_t>(kOverA ? static_cast<int64_t>(p + j) * N + n : n * R + p + j) * Factor<F>::kSize
                      : kNowhere;
        f[a][k] = Factor<F>::strided(rsrc, at);
      }
    }

  const int rp = pool.rp;
  const int64_t places = static_cast<int64_t>(plan.max_tiles) * kTile;
  for (int i = tid; i < kTile * 8 * KR; i += kThreads) {   // four ranks of a token
    const int tok = i / (8 * KR), p = i % (8 * KR) * 4;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (tok < t.count && p < rp) {
      const float* src = u.H + (place + tok) * rp + p;
      for (int q = 0; q < u.ks; ++q) x += *reinterpret_cast<const f32x4*>(src + q * places * rp);
    }
    bf16x4 h[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __bf16 piece[3];
      split3(x[j], piece);
#pragma unroll
      for (int q = 0; q < 3; ++q) h[q][j] = piece[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<bf16x4*>(&hs[q][tok][p]) = h[q];
  }
  __syncthreads();
  const float g = pool.gain * (pool.gains != nullptr ? pool.gains[t.slot] : 1.f);
  const uint64_t key = kOverA && u.drop.thr != 0 ? drop_key(u.drop) : 0;
  for (int m = 0; 16 * m < t.count; ++m) {
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
    store(m, true, g, key);
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
template <int NR, bool kRankMajor>
__device__ __forceinline__ void grad_job(const AdapterGrad& jb, uint32_t wg, const PlanView& plan, const Pool& pool,
                                         float (*part)[8 * (NR > 2 ? 2 : NR) * 4 * 64]) {
  constexpr int kParts = NR > 2 ? 2 : 1, NT = NR > 2 ? 2 : NR, kWaves = 4 / kParts;
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave % kParts, w = wave / kParts, tile0 = half * NT;
  const int64_t F = jb.F, places = static_cast<int64_t>(plan.max_tiles) * kTile;
  const uint32_t groups = static_cast<uint32_t>((F + 127) / 128);
  const int64_t group = wg % groups;
  const int at_chunk = wg / groups;
  const int4 info = *reinterpret_cast<const int4*>(plan.info);
  if (info.z != plan.n || info.w != plan.slots || at_chunk >= info.y) return;
  const int4 chunk = plan.chunks[at_chunk];
  const int slot = chunk.x, first = chunk.y, tiles = chunk.z;
  if (static_cast<unsigned>(slot) >= static_cast<unsigned>(plan.slots) || first < 0 || tiles < 1 || first + tiles > plan.max_tiles)
    return;
  const int64_t f0 = group * 128 + 8 * li, f = f0 < F ? f0 : F - 8;   // 8 | F
  const int steps = 2 * tiles - (tile_info(plan, first + tiles - 1).count > 32 ? 0 : 1);
  const uint32_t thr = kRankMajor ? jb.drop.thr : 0;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  f32x4 acc[8][NT];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t place0 = static_cast<int64_t>(first) * kTile + 8 * lg;
  u32x4 x[2][8], b[3][NT];
  int64_t token[2][8];
  auto load = [&](int set, int s) __attribute__((always_inline)) {
    if (s >= steps) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) token[set][i] = token_at(plan, place0 + 32 * static_cast<int64_t>(s) + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[set][i] = *reinterpret_cast<const u32x4*>(jb.L + token[set][i] * F + f);
  };
  auto load_s = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) {   // of an odd number of rank tiles the last half's second repeats the first
        const int tile = tile0 + t < NR ? tile0 + t : tile0;
        b[h][t] = *reinterpret_cast<const u32x4*>(jb.St + (h * 16 * NR + tile * 16 + li) * places + place0 + 32 * static_cast<int64_t>(s));
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
  const bool whole = chunk.w == 1;
  const int64_t nf = whole ? jb.nf : F;
  const int nr = whole ? pool.rank : 16 * NR;
  const float coef = whole ? pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f) : 1.f;
  float* o = whole ? jb.out + slot * (nf * nr) : jb.partials + at_chunk * (F * 16 * NR);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = coef * acc[j][t][v];
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

// job 0: dB over dY; job 1: dA over X
template <int NT>
__global__ __launch_bounds__(kThreads, 2) void grad_kernel(AdapterGradJobs jobs, PlanView plan, Pool pool, uint32_t first) {
  __shared__ float part[2][8 * (NT > 2 ? 2 : NT) * 4 * 64];
  if (blockIdx.x < first)
    grad_job<NT, false>(jobs.job[0], blockIdx.x, plan, pool, part);
  else
    grad_job<NT, true>(jobs.job[1], blockIdx.x - first, plan, pool, part);
}

// gain times the sum of a slot's partials in chunk order; zeros without tokens
__global__ __launch_bounds__(kThreads) void grad_sum_kernel(AdapterGradJobs jobs, PlanView plan, Pool pool, uint32_t first) {
  const bool rank_major = blockIdx.x >= first;
  const AdapterGrad& jb = jobs.job[rank_major ? 1 : 0];
  const int slot = blockIdx.y, R = pool.rank, rp = pool.rp;
  int chunk = 0, chunks = 0;
  if (plan.n > 0) {
    const int4 info = *reinterpret_cast<const int4*>(plan.info);
    if (info.z != plan.n || info.w != plan.slots) return;
    chunk = plan.slot_chunks[slot];
    chunks = plan.slot_chunks[slot + 1] - chunk;
    if (chunks == 1 || chunk < 0 || chunks < 0 || chunk + chunks > plan.max_chunks) return;
  }
  const int64_t i = static_cast<int64_t>(blockIdx.x - (rank_major ? first : 0)) * kThreads + threadIdx.x, nf = jb.nf;
  if (i >= nf * R) return;
  const int64_t at = rank_major ? i / nf * jb.F + i % nf : i / R * rp + i % R;
  float x = 0.f;
  for (int q = 0; q < chunks; ++q) x += jb.partials[(chunk + q) * (jb.F * rp) + at];
  const float g = pool.gain * (pool.gains != nullptr ? pool.gains[slot] : 1.f);
  jb.out[slot * (nf * R) + i] = chunks > 0 ? g * x : 0.f;
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

// K ranges for about m tiles' halves of tokens
int splits_for(int64_t halves, int64_t K) {
  // about a workgroup of eight waves per CU, each range with a step for every wave
  int64_t ks = 256 / halves;
  const int64_t most = (K + 31) / 32 / kDownWaves;
  if (ks > most) ks = most;
  return static_cast<int>(ks < 1 ? 1 : (ks > 16 ? 16 : ks));
}
// how many halves of tiles a batch may have, the slots' last ones half of the time
int64_t halves_of(int64_t n, int slots) { return 1 + n / 32 + (n < slots ? n : slots) / 2; }

}  // namespace

#define LQ_BY_RANK(rp, CALL) \
  switch ((rp) / 16) {       \
    case 1: CALL(1); break;  \
    case 2: CALL(2); break;  \
    case 3: CALL(3); break;  \
    default: CALL(4); break; \
  }

int adapters_down_splits(int64_t n, int slots, int64_t K) { return splits_for(halves_of(n, slots), K); }

int64_t adapters_down_tiles_bound(int64_t n, int slots, int64_t K) {
  int64_t bound = plan_layout(n, slots).max_tiles * adapters_down_splits(n, slots, K);
  for (int ks = adapters_down_splits(n, slots, K) + 1; ks <= adapters_down_splits(1, slots, K); ++ks) {
    // the most tokens that take as many ranges
    int64_t lo = 1, hi = n;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (adapters_down_splits(mid, slots, K) >= ks) lo = mid;
      else hi = mid - 1;
    }
    const int64_t tiles = plan_layout(lo, slots).max_tiles * adapters_down_splits(lo, slots, K);
    if (tiles > bound) bound = tiles;
  }
  return bound;
}

hipError_t launch_adapters_down(AdapterDownJobs jobs, const PlanView& plan, const Pool& pool, hipStream_t s) {
  for (AdapterDown& j : jobs.job) j.wgs = j.L != nullptr ? static_cast<unsigned>(2 * plan.max_tiles * j.ks) : 0;
  const dim3 grid(jobs.job[0].wgs + jobs.job[1].wgs);
#define LQ_DOWN(NT)                                                                                                             \
  do {                                                                                                                          \
    if (pool.dt == LOFTQ_BF16)                                                                                                  \
      LQ_LAUNCH("adapters_down", (down_kernel<NT, __bf16>), grid, dim3(kDownThreads), 0, s, jobs, plan, pool);                  \
    else                                                                                                                        \
      LQ_LAUNCH("adapters_down", (down_kernel<NT, float>), grid, dim3(kDownThreads), 0, s, jobs, plan, pool);                   \
  } while (0)
  LQ_BY_RANK(pool.rp, LQ_DOWN)
#undef LQ_DOWN
  return hipGetLastError();
}

hipError_t launch_adapters_sum(AdapterSumJobs jobs, const PlanView& plan, int rp, hipStream_t s) {
  LQ_LAUNCH("adapters_sum", sum_kernel, dim3(static_cast<unsigned>(2 * plan.max_tiles * (rp / 16)), 2), dim3(kThreads), 0, s,
            jobs, plan, rp);
  return hipGetLastError();
}

template <typename O, typename F, bool kOverA>
static void up_by_shape(const AdapterUp& u, const PlanView& plan, const Pool& pool, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((u.features + 255) / 256);
  const dim3 grid(static_cast<unsigned>(plan.max_tiles) * blocks), block(kThreads);
  const bool vec = u.features % (16 / static_cast<int64_t>(sizeof(O))) == 0;
  if (pool.rp <= 32) {
    if (vec) LQ_LAUNCH("adapters_up", (up_kernel<O, F, 1, true, kOverA>), grid, block, 0, s, u, plan, pool, blocks);
    else LQ_LAUNCH("adapters_up", (up_kernel<O, F, 1, false, kOverA>), grid, block, 0, s, u, plan, pool, blocks);
  } else {
    if (vec) LQ_LAUNCH("adapters_up", (up_kernel<O, F, 2, true, kOverA>), grid, block, 0, s, u, plan, pool, blocks);
    else LQ_LAUNCH("adapters_up", (up_kernel<O, F, 2, false, kOverA>), grid, block, 0, s, u, plan, pool, blocks);
  }
}

hipError_t launch_adapters_up(const AdapterUp& u, const PlanView& plan, const Pool& pool, hipStream_t s) {
#define LQ_UP(O, F)                                           \
  do {                                                        \
    if (u.over_a) up_by_shape<O, F, true>(u, plan, pool, s);  \
    else up_by_shape<O, F, false>(u, plan, pool, s);          \
  } while (0)
  if (u.odt == LOFTQ_BF16) {
    if (pool.dt == LOFTQ_BF16) LQ_UP(__bf16, __bf16);
    else LQ_UP(__bf16, float);
  } else {
    if (pool.dt == LOFTQ_BF16) LQ_UP(float, __bf16);
    else LQ_UP(float, float);
  }
#undef LQ_UP
  return hipGetLastError();
}

hipError_t launch_adapters_grad(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s) {
  unsigned wgs[2];
  for (int j = 0; j < 2; ++j) wgs[j] = static_cast<unsigned>((jobs.job[j].F + 127) / 128 * plan.max_chunks);
#define LQ_GRAD(NT) \
  LQ_LAUNCH("adapters_grad", (grad_kernel<NT>), dim3(wgs[0] + wgs[1]), dim3(kThreads), 0, s, jobs, plan, pool, wgs[0])
  LQ_BY_RANK(pool.rp, LQ_GRAD)
#undef LQ_GRAD
  return hipGetLastError();
}

hipError_t launch_adapters_grad_sum(const AdapterGradJobs& jobs, const PlanView& plan, const Pool& pool, hipStream_t s) {
  const unsigned first = blocks_for(jobs.job[0].nf * pool.rank), second = blocks_for(jobs.job[1].nf * pool.rank);
  LQ_LAUNCH("adapters_grad_sum", grad_sum_kernel, dim3(first + second, pool.slots), dim3(kThreads), 0, s, jobs, plan, pool, first);
  return hipGetLastError();
}

hipError_t launch_adapters_pad(const __bf16* in, __bf16* out, int64_t n, int64_t from, int64_t to, hipStream_t s) {
  LQ_LAUNCH("adapters_pad", pad_kernel, dim3(blocks_for(n * (to / 8))), dim3(kThreads), 0, s, in, out, n, from, to);
  return hipGetLastError();
}

}  // namespace loftq
