// Operands and thin products of the adapted layer's training path: the adapter's bf16
// operands, the base weight in bf16, X A^T and dY B (n x r), and the adapter's
// gradients (features x r) as products over the tokens.  A gradient needs two of each,
// over dY and over X: one launch takes both, as two jobs of one grid.
//
// All of it is bound by loads: the arithmetic of the thin products is a hundredth of the
// layer's.  Gradient of 2048 tokens x (11008 x 4096), r = 64: base and operands 36 us (25 MB
// of codes in, 90 MB of bf16 out), dY B and X A^T 33 us (their second operand, from L2,
// is as many bytes as four 16-token tiles of dY), their sums 8 us, dB and dA 27 us (62 MB of dY
// and X), their sums 6 us.  8192 tokens x (4096 x 11008), r = 16: 37, 81, 5, 47 and 5 us, X's
// mask being drawn twice.
//
// v_mfma_f32_16x16x32_bf16: lane L supplies A[L%16][8(L/16) + j] and
// B[8(L/16) + j][L%16] (j = 0..7) and receives D[4(L/16) + v][L%16] in element v.
#include "buffer.h"
#include "layer.h"

namespace loftq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---- what a call's products read, in one launch ----
// Work of thread i of the adapter's operands, eight elements each, zeros past r (and past
// `rows` in Bt).
__device__ __forceinline__ void adapter_operand(const AdapterOperands& a, uint32_t i) {
  const uint32_t cols = static_cast<uint32_t>(a.cols), rows = static_cast<uint32_t>(a.rows);
  const uint32_t rows_pad = static_cast<uint32_t>(a.rows_pad), groups = static_cast<uint32_t>(a.ld) / 8;
  bf16x8 o;
  if (a.Ab != nullptr) {
    const uint32_t per = cols / 8, n = a.rp * per;
    if (i < n) {
      const int p = i / per;
      const int64_t c = static_cast<int64_t>(i % per) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(p < a.r ? a.A[p * a.cols + c + j] : 0.f);
      *reinterpret_cast<bf16x8*>(a.Ab + p * a.cols + c) = o;
      return;
    }
    i -= n;
  }
  if (a.At != nullptr) {   // neighbouring threads take neighbouring columns, whose reads are one run
    const uint32_t n = groups * cols;
    if (i < n) {
      const int64_t c = i % cols;
      const int e = static_cast<int>(i / cols) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = (e + j) % a.rp;
        o[j] = static_cast<__bf16>(p < a.r && e < 3 * a.rp ? a.A[p * a.cols + c] : 0.f);
      }
      *reinterpret_cast<bf16x8*>(a.At + c * a.ld + e) = o;
      return;
    }
    i -= n;
  }
  if (a.Bb != nullptr) {
    const uint32_t n = groups * rows;
    if (i < n) {
      const int64_t row = i / groups;
      const int e = static_cast<int>(i % groups) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = (e + j) % a.rp;
        o[j] = static_cast<__bf16>(p < a.r && e < 3 * a.rp ? a.B[row * a.r + p] : 0.f);
      }
      *reinterpret_cast<bf16x8*>(a.Bb + row * a.ld + e) = o;
      return;
    }
    i -= n;
  }
  if (a.Bt != nullptr && i < a.rp * (rows_pad / 8)) {   // neighbouring threads take neighbouring ranks
    const int p = i % a.rp;
    const int64_t row = static_cast<int64_t>(i / a.rp) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = static_cast<__bf16>(p < a.r && row + j < a.rows ? a.B[(row + j) * a.r + p] : 0.f);
    *reinterpret_cast<bf16x8*>(a.Bt + p * a.rows_pad + row) = o;
  }
}

// A word of eight codes (the first in the high nibble of the low byte) and its scale as
// bf16(fp32 value).
__device__ __forceinline__ u32x4 decode8(const float* lvl, uint32_t word, float sc) {
  bf16x8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(lvl[word >> (8 * (j >> 1) + (j & 1 ? 0 : 4)) & 15u] * sc);
  return __builtin_bit_cast(u32x4, o);
}
// The codes and the scale of eight elements of a row from column c on (8 | c).
struct NfSource {
  const uint8_t* packed;
  const float* absmax;
  const int8_t* qabsmax;
  const float* dq_scale;
  __device__ __forceinline__ void fetch(int64_t e, uint32_t& word, float& sc) const {
    const int64_t b = e >> 6;
    word = *reinterpret_cast<const uint32_t*>(packed + (e >> 1));
    sc = qabsmax != nullptr ? static_cast<float>(qabsmax[b]) * dq_scale[b >> 8] : absmax[b];
  }
  __device__ __forceinline__ void fetch(int64_t row, int64_t c, int64_t rows, int64_t cols, uint32_t& word, float& sc) const {
    fetch(row * cols + c, word, sc);
  }
};
struct MxSource {
  const uint8_t* packed;
  const uint8_t* scales;
  __device__ __forceinline__ void fetch(int64_t row, int64_t c, int64_t rows, int64_t cols, uint32_t& word, float& sc) const {
    const int64_t steps = (cols + kMxStep - 1) / kMxStep;
    word = *reinterpret_cast<const uint32_t*>(packed + row * steps * (kMxStep / 2) + c / 2);
    sc = mx_scale(scales[(c / kMxStep * rows + row) * 8 + (c % kMxStep) / kMxBlock]);
  }
};
struct Levels {
  float v[16];
};

// One 64 x 128 tile of the base turned round in LDS: thread t decodes rows 2 (t / 8) and the
// next, columns 16 (t % 8) .. + 15, and keeps the two rows' values of a column in one word
// (row stride 33 words: a wave's 64 words fall into 64 banks); then the 8 lanes of a column
// write its 64 rows, a line.
constexpr int kTurnRows = 64, kTurnCols = 128;
template <typename Src>
__device__ __forceinline__ void turn_base(const Src& src, const float* lvl, uint32_t (*tile)[33], int64_t tr, int64_t tc,
                                          int64_t rows, int64_t cols, int64_t rows_pad, __bf16* __restrict__ out) {
  const int tid = threadIdx.x, pair = tid / 8, c16 = (tid % 8) * 16;
  const int64_t row = tr * kTurnRows + 2 * pair;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  uint32_t word[2][2];
  float sc[2][2];
  bool live[2][2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // every load in flight before the first is decoded
      const int64_t c = tc * kTurnCols + c16 + q * 8;
      live[q][h] = row + h < rows && c < cols;
      src.fetch(live[q][h] ? row + h : 0, live[q][h] ? c : 0, rows, cols, word[q][h], sc[q][h]);
    }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const u32x4 lo = live[q][0] ? decode8(lvl, word[q][0], sc[q][0]) : zero;
    const u32x4 hi = live[q][1] ? decode8(lvl, word[q][1], sc[q][1]) : zero;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      tile[c16 + q * 8 + j][pair] = __builtin_amdgcn_perm(hi[j >> 1], lo[j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
  }
  __syncthreads();
  // 16 bytes of 4 rows' pairs a store, the 8 lanes of a column one run of 128 bytes
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int cc = q * 32 + tid / 8, w0 = (tid % 8) * 4;
    const int64_t c = tc * kTurnCols + cc;
    if (c >= cols) continue;
    const u32x4 v = {tile[cc][w0], tile[cc][w0 + 1], tile[cc][w0 + 2], tile[cc][w0 + 3]};
    *reinterpret_cast<u32x4*>(out + c * rows_pad + tr * kTurnRows + 2 * w0) = v;
  }
}

// Workgroups 0 .. base_wgs - 1 form the base's operand (transposed, as it lies, or, over
// MXFP4, the codes of X), the next operand_wgs the adapter's, the rest pads dY's rows.
template <typename Src, int kBase>   // kBase 0: as it lies, 1: transposed, 2: MXFP4 codes of `x`
__global__ __launch_bounds__(kThreads) void prepare_kernel(Src src, Levels lv, PrepareArgs p) {
  __shared__ float lvl[16];
  __shared__ uint32_t tile[kBase == 1 ? kTurnCols : 1][33];
  const int tid = threadIdx.x;
  uint32_t wg = blockIdx.x;
  if (wg < p.base_wgs) {
    if constexpr (kBase == 2) {
      const uint32_t id = wg * kThreads + tid, per_row = static_cast<uint32_t>(p.steps * (kMxStep / 8));
      const int64_t row = id / per_row, c0 = static_cast<int64_t>(id % per_row) * 8;
      if (row >= p.n) return;   // whole quads: per_row % 32 == 0
      float x[8];
      const bf16x8 v = c0 < p.a.cols ? *reinterpret_cast<const bf16x8*>(p.x + row * p.a.cols + c0) : bf16x8{};
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(v[j]);
      uint32_t byte;
      reinterpret_cast<uint32_t*>(p.xq)[id] = mx_encode8(x, byte);
      if ((tid & 3) == 0) p.xs[(c0 / kMxStep * p.n + row) * 8 + (c0 % kMxStep) / kMxBlock] = static_cast<uint8_t>(byte);
    } else {
      if (tid < 16) lvl[tid] = lv.v[tid];
      __syncthreads();
      if constexpr (kBase == 1) {
        const uint32_t ntr = static_cast<uint32_t>(p.a.rows_pad / kTurnRows);
        turn_base(src, lvl, tile, wg % ntr, wg / ntr, p.a.rows, p.a.cols, p.a.rows_pad, p.base);
      } else {
        // four groups of eight a thread, every load in flight before the first is decoded
        const int64_t n = p.a.rows * p.a.cols, e0 = (static_cast<int64_t>(wg) * (4 * kThreads) + tid) * 8;
        uint32_t word[4];
        float sc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t e = e0 + q * (kThreads * 8);
          src.fetch(e < n ? e : 0, word[q], sc[q]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t e = e0 + q * (kThreads * 8);
          if (e < n) *reinterpret_cast<u32x4*>(p.base + e) = decode8(lvl, word[q], sc[q]);
        }
      }
    }
    return;
  }
  wg -= p.base_wgs;
  if (wg < p.operand_wgs) {
    adapter_operand(p.a, wg * kThreads + tid);
    return;
  }
  wg -= p.operand_wgs;
  const uint32_t id = wg * kThreads + tid, per_row = static_cast<uint32_t>(p.a.rows_pad / 8);
  const int64_t row = id / per_row, c = static_cast<int64_t>(id % per_row) * 8;
  if (row >= p.n) return;
  bf16x8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = c + j < p.a.rows ? p.x[row * p.a.rows + c + j] : static_cast<__bf16>(0.f);
  *reinterpret_cast<bf16x8*>(p.padded + row * p.a.rows_pad + c) = o;
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

// ---- thin product over the features: partial q of keep(X) M^T over the q-th K range ----
// A workgroup takes 32 tokens and one range, which its four waves share U steps of 32 at a
// time; M (rank-major, K along its rows) serves both 16-token tiles.  All loads of U steps
// are issued before the first product.  The waves' sums meet in LDS.
template <int NT>
__global__ __launch_bounds__(kThreads) void down_kernel(DownJobs jobs, int64_t n) {
  constexpr int U = NT <= 2 ? 4 : 2;
  __shared__ float part[3][2 * NT * 4 * 64];
  const DownJob& jb = jobs.job[blockIdx.x < jobs.job[0].wgs ? 0 : 1];
  const uint32_t wg = blockIdx.x < jobs.job[0].wgs ? blockIdx.x : blockIdx.x - jobs.job[0].wgs;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), li = lane & 15, lg = lane >> 4;
  const int64_t K = jb.K, m0 = static_cast<int64_t>(wg / jb.ks) * 32;
  const int q = wg % jb.ks, steps = static_cast<int>(K / 32), per = (steps + jb.ks - 1) / jb.ks;
  const int begin = __builtin_amdgcn_readfirstlane(q * per), end = begin + per < steps ? begin + per : steps;
  const uint32_t thr = jb.drop.thr;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  // this lane's offsets from a step's first bytes; tokens past the last and steps past the
  // range are zeros
  uint32_t xat[2], bat[NT];
#pragma unroll
  for (int t = 0; t < 2; ++t) xat[t] = static_cast<uint32_t>(((t * 16 + li) * K + 8 * lg) * 2);
#pragma unroll
  for (int p = 0; p < NT; ++p) bat[p] = static_cast<uint32_t>(((p * 16 + li) * K + 8 * lg) * 2);
  f32x4 acc[2][NT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int p = 0; p < NT; ++p) acc[t][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = begin + w * U; s0 < end; s0 += 4 * U) {
    u32x4 x[U][2], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = static_cast<int64_t>(s0 + u) * 32;
      const bool any = s0 + u < end;
      const __amdgpu_buffer_rsrc_t xb = buffer_of(jb.X + m0 * K + k, any ? ((n - m0) * K - k) * 2 : 0);
      const __amdgpu_buffer_rsrc_t bb = buffer_at(jb.M + k, any);
#pragma unroll
      for (int t = 0; t < 2; ++t) x[u][t] = __builtin_amdgcn_raw_buffer_load_b128(xb, xat[t], 0, 0);
#pragma unroll
      for (int p = 0; p < NT; ++p) b[u][p] = __builtin_amdgcn_raw_buffer_load_b128(bb, bat[p], 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4 v = x[u][t];
        if (thr != 0)
          v = drop8(v, key, static_cast<uint64_t>((m0 + 16 * t + li) * K + static_cast<int64_t>(s0 + u) * 32 + 8 * lg), thr);
#pragma unroll
        for (int p = 0; p < NT; ++p) acc[t][p] = mfma16(v, b[u][p], acc[t][p]);
      }
    }
  }
  if (w > 0)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int p = 0; p < NT; ++p)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[w - 1][((t * NT + p) * 4 + v) * 64 + lane] = acc[t][p][v];
  __syncthreads();
  if (w > 0) return;
  float* o = jb.out + static_cast<int64_t>(q) * n * (16 * NT);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int p = 0; p < NT; ++p)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t mm = m0 + 16 * t + 4 * lg + v;
        const int at = ((t * NT + p) * 4 + v) * 64 + lane;
        const float y = ((acc[t][p][v] + part[0][at]) + part[1][at]) + part[2][at];
        if (mm < n) o[mm * (16 * NT) + p * 16 + li] = y;
      }
}

// The sum of the partials in split order, as three bf16 pieces x = h0 + h1 + h2 (each the
// rounding of what the ones before leave: the three hold 24 bits, so the products they
// enter lose nothing against fp32; an infinity or NaN is all in the first).  Ranks past r
// and tokens past n are zeros.  A workgroup takes 32 tokens and 16 ranks; the rank-major
// form is turned round in LDS.
__device__ __forceinline__ void split3(float x, __bf16 (&h)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    h[q] = static_cast<__bf16>(x);
    x = __builtin_isfinite(static_cast<float>(h[q])) ? x - static_cast<float>(h[q]) : 0.f;
  }
}
__global__ __launch_bounds__(kThreads) void down_sum_kernel(DownSumJobs jobs, int64_t n, int r, int rp, int ld,
                                                            int64_t n_pad) {
  __shared__ __align__(4) __bf16 turned[3 * 16][32 + 2];
  const DownSumJob& jb = jobs.job[blockIdx.x < jobs.job[0].wgs ? 0 : 1];
  const uint32_t wg = blockIdx.x < jobs.job[0].wgs ? blockIdx.x : blockIdx.x - jobs.job[0].wgs;
  const int parts = rp / 16, p0 = static_cast<int>(wg % parts) * 16;
  const int64_t m0 = static_cast<int64_t>(wg / parts) * 32;
#pragma unroll
  for (int i = threadIdx.x; i < 32 * 16; i += kThreads) {
    const int tok = i / 16, p = p0 + i % 16;
    const int64_t m = m0 + tok;
    float x = 0.f;
    if (m < n && p < r) {
      const float* src = jb.partials + m * rp + p;
      int q = 0;
      for (; q + 4 <= jb.ks; q += 4) {   // four loads in flight, added in order
        const float a = src[q * n * rp], b = src[(q + 1) * n * rp], c = src[(q + 2) * n * rp], d = src[(q + 3) * n * rp];
        x = (((x + a) + b) + c) + d;
      }
      for (; q < jb.ks; ++q) x += src[q * n * rp];
    }
    __bf16 h[3];
    if (jb.S != nullptr && m < n) {
      split3(jb.gain * x, h);
#pragma unroll
      for (int q = 0; q < 3; ++q) jb.S[m * ld + q * rp + p] = h[q];
      if (p < ld - 3 * rp) jb.S[m * ld + 3 * rp + p] = static_cast<__bf16>(0.f);   // ld - 3 rp is rp or 0
    }
    if (jb.St != nullptr) {
      split3(x, h);
#pragma unroll
      for (int q = 0; q < 3; ++q) turned[q * 16 + i % 16][tok] = h[q];
    }
  }
  if (jb.St == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * 16 * 16; i += kThreads) {   // two tokens a store
    const int row = i / 16, t = (i % 16) * 2;
    *reinterpret_cast<uint32_t*>(jb.St + (row / 16 * rp + p0 + row % 16) * n_pad + m0 + t) =
        *reinterpret_cast<const uint32_t*>(&turned[row][t]);
  }
}

// ---- thin product over the tokens: the adapter's gradients ----
// out[i][p] = sum_t keep(L)[t][i] S[t][p].  The matrix cores want each operand's K (tokens) in
// one lane, and L's tokens are rows: lane L loads 8 tokens x 8 features (16 bytes of 8
// rows) and turns the 8 x 8 block round in its registers, which gives the operands of 8
// products, the j-th for features 8 (L%16) + j.  A workgroup takes 128 features and a token
// range, which its four waves share 32 tokens at a time, the next step's rows of L in flight
// while one is multiplied; past 32 ranks two waves share a step, half of the ranks each (the
// sums of all of them leave a wave no registers for its loads).  S's operands are loaded when
// their step begins: ahead of it they cost the second wave per SIMD (38 against 27 us at 2048
// tokens of 11008 and 4096 features, r = 64).  The sums meet in LDS.  kRankMajor (dA): S is the first operand, so a
// lane holds 8 consecutive features of a rank; else (dB) a lane's rank is L%16.
template <int NR, bool kRankMajor>
__device__ __forceinline__ void grad_job(const GradJob& jb, uint32_t wg, int64_t n, int64_t n_pad, int r,
                                         float (*part)[8 * (NR > 2 ? 2 : NR) * 4 * 64]) {
  constexpr int kParts = NR > 2 ? 2 : 1, NT = NR > 2 ? 2 : NR, kWaves = 4 / kParts;   // waves per step's ranks, of a rank half
  const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = wave % kParts, w = wave / kParts, tile0 = half * NT;
  const int64_t group = wg / jb.ts, F = jb.F;
  const int q = wg % jb.ts;
  const int64_t f0 = group * 128 + 8 * li, f = f0 < F ? f0 : F - 8;   // F % 8 == 0
  const int steps = static_cast<int>(n_pad / 32), per = (steps + jb.ts - 1) / jb.ts;
  const int begin = q * per, end = begin + per < steps ? begin + per : steps;
  const uint32_t thr = kRankMajor ? jb.drop.thr : 0;
  const uint64_t key = thr != 0 ? drop_key(jb.drop) : 0;
  f32x4 acc[8][NT];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this lane's offsets from a step's first bytes; tokens past the last are zeros
  uint32_t xat[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) xat[i] = static_cast<uint32_t>(((8 * lg + i) * F + f) * 2);
  const uint32_t bat = static_cast<uint32_t>((li * n_pad + 8 * lg) * 2);
  u32x4 x[2][8], b[3][NT];
  auto load = [&](int set, int s) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(s) * 32;
    const __amdgpu_buffer_rsrc_t xb = buffer_of(jb.L + t0 * F, s < end ? (n - t0) * F * 2 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[set][i] = __builtin_amdgcn_raw_buffer_load_b128(xb, xat[i], 0, 0);
  };
  auto load_s = [&](int s) __attribute__((always_inline)) {
    const int64_t t0 = static_cast<int64_t>(s) * 32;
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) {   // of an odd number of rank tiles the last half's second repeats the first
        const int tile = tile0 + t < NR ? tile0 + t : tile0;
        b[h][t] = __builtin_amdgcn_raw_buffer_load_b128(
            buffer_at(jb.St + static_cast<int64_t>(h * 16 * NR + tile * 16) * n_pad + t0, s < end), bat, 0, 0);
      }
  };
  auto multiply = [&](int set, int s) __attribute__((always_inline)) {
    if (thr != 0)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[set][i] = drop8(x[set][i], key, static_cast<uint64_t>((static_cast<int64_t>(s) * 32 + 8 * lg + i) * F + f), thr);
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
          acc[2 * c][t] = kRankMajor ? mfma16(b[h][t], lo, acc[2 * c][t])
                                     : mfma16(lo, b[h][t], acc[2 * c][t]);
          acc[2 * c + 1][t] =
              kRankMajor ? mfma16(b[h][t], hi, acc[2 * c + 1][t])
                         : mfma16(hi, b[h][t], acc[2 * c + 1][t]);
        }
    }
  };
  if (begin + w < end) {
    load(0, begin + w);
    for (int s = begin + w; s < end; s += 2 * kWaves) {
      load_s(s);
      load(1, s + kWaves);
      multiply(0, s);
      if (s + kWaves >= end) break;
      load_s(s + kWaves);
      load(0, s + 2 * kWaves);
      multiply(1, s + kWaves);
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
  // one range: the gradient itself; more: a partial sum with whole padded ranks and features
  const bool whole = jb.ts == 1;
  const int64_t nf = whole ? jb.nf : F;
  const int nr = whole ? r : 16 * NR;
  const float coef = whole ? jb.coef : 1.f;
  float* o = whole ? jb.out : jb.partials + static_cast<int64_t>(q) * F * (16 * NR);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = coef * acc[j][t][v];
      if constexpr (kRankMajor) {
        const int p = (tile0 + t) * 16 + 4 * lg + v;   // features f0 .. f0 + 7
        if (p < nr && f0 < F)                // nf == F here, and 8 | F
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
__global__ __launch_bounds__(kThreads, 2) void grad_kernel(GradJobs jobs, int64_t n, int64_t n_pad, int r) {
  __shared__ float part[2][8 * (NT > 2 ? 2 : NT) * 4 * 64];
  if (blockIdx.x < jobs.job[0].wgs)
    grad_job<NT, false>(jobs.job[0], blockIdx.x, n, n_pad, r, part);
  else
    grad_job<NT, true>(jobs.job[1], blockIdx.x - jobs.job[0].wgs, n, n_pad, r, part);
}

// coef times the sum of the partials in range order; job 0 feature-major, job 1 rank-major
__global__ __launch_bounds__(kThreads) void grad_sum_kernel(GradJobs jobs, int r, int rp) {
  const uint32_t first = (static_cast<uint32_t>(jobs.job[0].nf) * r + kThreads - 1) / kThreads;
  const bool rank_major = blockIdx.x >= first;
  const GradJob& jb = jobs.job[rank_major ? 1 : 0];
  const uint32_t i = (blockIdx.x - (rank_major ? first : 0)) * kThreads + threadIdx.x, nf = static_cast<uint32_t>(jb.nf);
  if (i >= nf * r) return;
  const int64_t at = rank_major ? i / nf * jb.F + i % nf : static_cast<int64_t>(i / r) * rp + i % r;
  float x = 0.f;
  for (int q = 0; q < jb.ts; ++q) x += jb.partials[q * jb.F * rp + at];
  jb.out[i] = jb.coef * x;
}

unsigned blocks_for(int64_t threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

Levels base_levels(const Base4& b) {
  Levels lv{};
  if (b.mx != nullptr) {
    const float mag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
    for (int i = 0; i < 16; ++i) lv.v[i] = i < 8 ? mag[i] : -mag[i - 8];
  } else {
    for (int i = 0; i < 16; ++i) lv.v[i] = nf_tables(b.bits).level[i];
  }
  return lv;
}

}  // namespace

hipError_t launch_prepare(PrepareArgs p, const Base4& b, PrepareBase kind, hipStream_t s) {
  const AdapterOperands& a = p.a;
  p.operand_wgs = a.r == 0 ? 0 : blocks_for((a.Ab ? a.rp * (a.cols / 8) : 0) + (a.Bt ? a.rp * (a.rows_pad / 8) : 0) +
                                            a.ld / 8 * ((a.At ? a.cols : 0) + (a.Bb ? a.rows : 0)));
  p.base_wgs = kind == kBaseNone         ? 0
               : kind == kBaseTransposed ? static_cast<unsigned>((a.rows_pad / kTurnRows) * ((a.cols + kTurnCols - 1) / kTurnCols))
               : kind == kBaseCodesOfX   ? blocks_for(p.n * p.steps * (kMxStep / 8))
                                         : blocks_for((a.rows * a.cols + 31) / 32);
  const unsigned pad_wgs = p.padded != nullptr ? blocks_for(p.n * (a.rows_pad / 8)) : 0;
  const dim3 grid(p.base_wgs + p.operand_wgs + pad_wgs);
  if (grid.x == 0) return hipSuccess;
  const Levels lv = base_levels(b);
  const NfSource nf{b.packed, b.absmax, b.qabsmax, b.dq_scale};
  const MxSource mx{b.packed, b.mx};
  if (kind == kBaseCodesOfX)
    LQ_LAUNCH("prepare_layer", (prepare_kernel<MxSource, 2>), grid, dim3(kThreads), 0, s, mx, lv, p);
  else if (kind == kBaseAsItLies || kind == kBaseNone)
    LQ_LAUNCH("prepare_layer", (prepare_kernel<NfSource, 0>), grid, dim3(kThreads), 0, s, nf, lv, p);
  else if (b.mx != nullptr)
    LQ_LAUNCH("prepare_layer", (prepare_kernel<MxSource, 1>), grid, dim3(kThreads), 0, s, mx, lv, p);
  else
    LQ_LAUNCH("prepare_layer", (prepare_kernel<NfSource, 1>), grid, dim3(kThreads), 0, s, nf, lv, p);
  return hipGetLastError();
}

#define LQ_BY_RANK(rp, CALL) \
  switch ((rp) / 16) {       \
    case 1: CALL(1); break;  \
    case 2: CALL(2); break;  \
    case 3: CALL(3); break;  \
    default: CALL(4); break; \
  }

int down_splits(int64_t n, int64_t K) {
  // about four workgroups per CU, each with at least 8 steps (two per wave)
  const int64_t groups = n > 32 ? (n + 31) / 32 : 1;
  int64_t ks = 1024 / groups;
  if (ks > K / 32 / 8) ks = K / 32 / 8;
  return static_cast<int>(ks < 1 ? 1 : (ks > 32 ? 32 : ks));
}

// Fewer tokens may be divided into more ranges: k ranges are taken up to 1024 / k groups.
int64_t down_rows_bound(int64_t n, int64_t K) {
  int64_t most = n;
  for (int64_t k = down_splits(0, K); k > 1; --k) {
    const int64_t tokens = 1024 / k * 32, rows = k * (tokens < n ? tokens : n);
    if (rows > most) most = rows;
  }
  return most;
}

hipError_t launch_down(DownJobs jobs, int64_t n, int rp, hipStream_t s) {
  for (DownJob& j : jobs.job) j.wgs = j.X != nullptr ? static_cast<unsigned>((n + 31) / 32 * j.ks) : 0;
  const dim3 grid(jobs.job[0].wgs + jobs.job[1].wgs);
#define LQ_DOWN(NT) LQ_LAUNCH("adapter_down", (down_kernel<NT>), grid, dim3(kThreads), 0, s, jobs, n)
  LQ_BY_RANK(rp, LQ_DOWN)
#undef LQ_DOWN
  return hipGetLastError();
}

hipError_t launch_down_sum(DownSumJobs jobs, int64_t n, int r, int rp, hipStream_t s) {
  for (DownSumJob& j : jobs.job) j.wgs = j.partials != nullptr ? static_cast<unsigned>((n + 31) / 32 * (rp / 16)) : 0;
  LQ_LAUNCH("adapter_down_sum", down_sum_kernel, dim3(jobs.job[0].wgs + jobs.job[1].wgs), dim3(kThreads), 0, s, jobs, n, r,
            rp, adapter_ld(rp), (n + 31) / 32 * 32);
  return hipGetLastError();
}

int grad_splits(int64_t n, int64_t rows_pad, int64_t cols) {
  // about two workgroups per CU for the two gradients, each with at least 128 tokens
  const int64_t groups = (rows_pad + 127) / 128 + (cols + 127) / 128;
  int64_t ts = groups > 0 ? 512 / groups : 1;
  const int64_t most = (n + 127) / 128;
  if (ts > most) ts = most;
  return static_cast<int>(ts < 1 ? 1 : (ts > 16 ? 16 : ts));
}

hipError_t launch_grad(GradJobs jobs, int64_t n, int r, int rp, hipStream_t s) {
  for (GradJob& j : jobs.job) j.wgs = static_cast<unsigned>((j.F + 127) / 128 * j.ts);
  const dim3 grid(jobs.job[0].wgs + jobs.job[1].wgs);
#define LQ_GRAD(NT) \
  LQ_LAUNCH("adapter_grad", (grad_kernel<NT>), grid, dim3(kThreads), 0, s, jobs, n, (n + 31) / 32 * 32, r)
  LQ_BY_RANK(rp, LQ_GRAD)
#undef LQ_GRAD
  return hipGetLastError();
}

hipError_t launch_grad_sum(const GradJobs& jobs, int r, int rp, hipStream_t s) {
  const dim3 grid(blocks_for(jobs.job[0].nf * r) + blocks_for(jobs.job[1].nf * r));
  LQ_LAUNCH("adapter_grad_sum", grad_sum_kernel, grid, dim3(kThreads), 0, s, jobs, r, rp);
  return hipGetLastError();
}

}  // namespace loftq
