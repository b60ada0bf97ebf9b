// Operands and thin products of the adapted layer's training path: the adapter's bf16
// operands, the base weight in bf16, X A^T and dY B (n x r), and the adapter's
// gradients (features x r) as products over the tokens.
//
// v_mfma_f32_16x16x32_bf16: lane L supplies A[L%16][8(L/16) + j] and
// B[8(L/16) + j][L%16] (j = 0..7) and receives D[4(L/16) + v][L%16] in element v.
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

// ---- the adapter's bf16 operands, zero past r (and past `rows` in Bt) ----
__global__ __launch_bounds__(kThreads) void adapter_operands_kernel(AdapterOperands a) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t nAb = a.rp * a.cols, nAt = a.ld * a.cols, nBb = a.ld * a.rows, nBt = a.rp * a.rows_pad;
  if (a.Ab != nullptr) {
    if (i < nAb) {
      const int64_t p = i / a.cols;
      a.Ab[i] = static_cast<__bf16>(p < a.r ? a.A[i] : 0.f);
      return;
    }
    i -= nAb;
  }
  if (a.At != nullptr) {
    if (i < nAt) {
      const int64_t c = i / a.ld, e = i - c * a.ld, p = e % a.rp;
      a.At[i] = static_cast<__bf16>(p < a.r && e < 3 * a.rp ? a.A[p * a.cols + c] : 0.f);
      return;
    }
    i -= nAt;
  }
  if (a.Bb != nullptr) {
    if (i < nBb) {
      const int64_t row = i / a.ld, e = i - row * a.ld, p = e % a.rp;
      a.Bb[i] = static_cast<__bf16>(p < a.r && e < 3 * a.rp ? a.B[row * a.r + p] : 0.f);
      return;
    }
    i -= nBb;
  }
  if (a.Bt != nullptr && i < nBt) {
    const int64_t p = i / a.rows_pad, row = i - p * a.rows_pad;
    a.Bt[i] = static_cast<__bf16>(p < a.r && row < a.rows ? a.B[row * a.r + p] : 0.f);
  }
}

// ---- the base weight in bf16 ----
// Both sources give 8 consecutive elements of a row (c % 8 == 0) as bf16(fp32 value).
struct NfSource {
  const uint8_t* packed;
  const float* absmax;
  const int8_t* qabsmax;
  const float* dq_scale;
  __device__ __forceinline__ u32x4 load8(const float* lvl, int64_t row, int64_t c, int64_t rows, int64_t cols) const {
    const int64_t e = row * cols + c, b = e >> 6;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(packed + (e >> 1));
    const float sc = qabsmax != nullptr ? static_cast<float>(qabsmax[b]) * dq_scale[b >> 8] : absmax[b];
    bf16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(lvl[word >> (8 * (j >> 1) + (j & 1 ? 0 : 4)) & 15u] * sc);
    return __builtin_bit_cast(u32x4, o);
  }
};
struct MxSource {
  const uint8_t* packed;
  const uint8_t* scales;
  __device__ __forceinline__ u32x4 load8(const float* lvl, int64_t row, int64_t c, int64_t rows, int64_t cols) const {
    const int64_t steps = (cols + kMxStep - 1) / kMxStep;
    const uint32_t word = *reinterpret_cast<const uint32_t*>(packed + row * steps * (kMxStep / 2) + c / 2);
    const float sc = mx_scale(scales[(c / kMxStep * rows + row) * 8 + (c % kMxStep) / kMxBlock]);
    bf16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = static_cast<__bf16>(lvl[word >> (8 * (j >> 1) + (j & 1 ? 0 : 4)) & 15u] * sc);
    return __builtin_bit_cast(u32x4, o);
  }
};
struct Levels {
  float v[16];
};

template <typename Src>
__global__ __launch_bounds__(kThreads) void base_bf16_kernel(Src src, Levels lv, int64_t rows, int64_t cols,
                                                             __bf16* __restrict__ out) {
  __shared__ float lvl[16];
  if (threadIdx.x < 16) lvl[threadIdx.x] = lv.v[threadIdx.x];
  __syncthreads();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 8;
  if (i >= rows * cols) return;
  const int64_t row = i / cols;
  *reinterpret_cast<u32x4*>(out + i) = src.load8(lvl, row, i - row * cols, rows, cols);
}

// One 64 x 64 tile per workgroup, turned round in LDS: thread t reads row t / 4, 16
// columns, and writes column t / 4, 16 rows.
template <typename Src>
__global__ __launch_bounds__(kThreads) void base_bf16_t_kernel(Src src, Levels lv, int64_t rows, int64_t cols,
                                                               int64_t rows_pad, __bf16* __restrict__ out) {
  __shared__ float lvl[16];
  __shared__ __align__(16) uint16_t tile[64][64 + 8];
  const int tid = threadIdx.x;
  if (tid < 16) lvl[tid] = lv.v[tid];
  __syncthreads();
  const int64_t ntr = rows_pad / 64;
  const int64_t tr = blockIdx.x % ntr, tc = blockIdx.x / ntr;
  const int64_t row = tr * 64 + tid / 4;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int cc = (tid % 4) * 16 + q * 8;
    const int64_t c = tc * 64 + cc;
    const u32x4 v = row < rows && c < cols ? src.load8(lvl, row, c, rows, cols) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[cc + j][tid / 4] = static_cast<uint16_t>(v[j >> 1] >> (16 * (j & 1)));
  }
  __syncthreads();
  const int64_t c = tc * 64 + tid / 4;
  if (c >= cols) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int rr = (tid % 4) * 16 + q * 8;
    *reinterpret_cast<u32x4*>(out + c * rows_pad + tr * 64 + rr) = *reinterpret_cast<const u32x4*>(&tile[tid / 4][rr]);
  }
}

__global__ __launch_bounds__(kThreads) void pad_rows_kernel(const __bf16* __restrict__ src, int64_t n, int64_t cols,
                                                            int64_t ld, __bf16* __restrict__ dst) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 8;
  if (i >= n * ld) return;
  const int64_t row = i / ld, c = i - row * ld;
  bf16x8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = c + j < cols ? src[row * cols + c + j] : static_cast<__bf16>(0.f);
  *reinterpret_cast<bf16x8*>(dst + i) = o;
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
// One wave per 16 tokens and range; M (rank-major, K along its rows) is shared by the
// four waves of a workgroup through the caches.  U steps of 32 are loaded before the
// first product; steps past the range repeat its last one with the tokens zeroed.
template <int NT, bool kDrop>
__global__ __launch_bounds__(kThreads) void down_kernel(const __bf16* __restrict__ X, int64_t n, int64_t K,
                                                        const __bf16* __restrict__ Mb, int ks, DropArg d,
                                                        float* __restrict__ out) {
  constexpr int U = NT <= 2 ? 4 : 2;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
  const int64_t group = blockIdx.x / ks;
  const int q = static_cast<int>(blockIdx.x - group * ks);
  const int64_t m0 = group * 64 + w * 16;
  if (m0 >= n) return;
  const int64_t m = m0 + li < n ? m0 + li : n - 1;
  const int64_t steps = K / 32, per = (steps + ks - 1) / ks;
  const int64_t begin = q * per, end = begin + per < steps ? begin + per : steps;
  const uint64_t key = kDrop ? drop_key(d) : 0;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t s0 = begin; s0 < end; s0 += U) {
    u32x4 x[U], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (s0 + u < end ? s0 + u : end - 1) * 32 + 8 * lg;
      x[u] = *reinterpret_cast<const u32x4*>(X + m * K + k);
#pragma unroll
      for (int t = 0; t < NT; ++t) b[u][t] = *reinterpret_cast<const u32x4*>(Mb + (t * 16 + li) * K + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (s0 + u < end ? s0 + u : end - 1) * 32 + 8 * lg;
      u32x4 v = s0 + u < end ? x[u] : u32x4{0u, 0u, 0u, 0u};
      if (kDrop) v = drop8(v, key, static_cast<uint64_t>(m * K + k), d.thr);
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = mfma16(v, b[u][t], acc[t]);
    }
  }
  float* o = out + static_cast<int64_t>(q) * n * (16 * NT);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t mm = m0 + 4 * lg + v;
      if (mm < n) o[mm * (16 * NT) + t * 16 + li] = acc[t][v];
    }
}

// The sum of the partials in split order, as three bf16 pieces x = h0 + h1 + h2 (each the
// rounding of what the ones before leave: the three hold 24 bits, so the products they
// enter lose nothing against fp32; an infinity or NaN is all in the first).  Ranks past r
// and tokens past n are zeros.
__device__ __forceinline__ void split3(float x, __bf16 (&h)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    h[q] = static_cast<__bf16>(x);
    x = __builtin_isfinite(static_cast<float>(h[q])) ? x - static_cast<float>(h[q]) : 0.f;
  }
}
__global__ __launch_bounds__(kThreads) void down_sum_kernel(const float* __restrict__ partials, int64_t n, int r, int rp,
                                                            int ks, float gain, int ld, __bf16* __restrict__ S,
                                                            __bf16* __restrict__ St, int64_t n_pad) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n_pad * rp) return;
  const int64_t p = i / n_pad, m = i - p * n_pad;
  float x = 0.f;
  if (m < n && p < r)
    for (int q = 0; q < ks; ++q) x += partials[(q * n + m) * rp + p];
  __bf16 h[3];
  if (S != nullptr && m < n) {
    split3(gain * x, h);
#pragma unroll
    for (int q = 0; q < 3; ++q) S[m * ld + q * rp + p] = h[q];
    if (p < ld - 3 * rp) S[m * ld + 3 * rp + p] = static_cast<__bf16>(0.f);   // ld - 3 rp is rp or 0
  }
  if (St != nullptr) {
    split3(x, h);
#pragma unroll
    for (int q = 0; q < 3; ++q) St[(q * rp + p) * n_pad + m] = h[q];
  }
}

// ---- thin product over the tokens: the adapter's gradients ----
// out[i][p] = sum_t L[t][i] S[t][p].  The matrix cores want each operand's K (tokens) in
// one lane, and L's tokens are rows: lane L loads 8 tokens x 8 features (16 bytes of 8
// rows) and turns the 8 x 8 block round in its registers, which gives the operands of 8
// products, the j-th for features 8 (L%16) + j.  A workgroup takes 128 features; its four
// waves share a token range 32 tokens at a time, and their sums meet in LDS.
template <int NT, bool kDrop>
__global__ __launch_bounds__(kThreads) void grad_kernel(const __bf16* __restrict__ L, int64_t n, int64_t F,
                                                        const __bf16* __restrict__ St, int64_t n_pad, int ts, DropArg d,
                                                        float* __restrict__ out) {
  __shared__ float part[2][8 * NT * 4 * 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
  const int64_t group = blockIdx.x / ts;
  const int q = static_cast<int>(blockIdx.x - group * ts);
  const int64_t f0 = group * 128 + 8 * li, f = f0 < F ? f0 : F - 8;   // F % 8 == 0
  const int64_t steps = n_pad / 32, per = (steps + ts - 1) / ts;
  const int64_t begin = q * per, end = begin + per < steps ? begin + per : steps;
  const uint64_t key = kDrop ? drop_key(d) : 0;
  f32x4 acc[8][NT];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t s = begin + w; s < end; s += 4) {
    const int64_t t0 = s * 32 + 8 * lg;
    u32x4 x[8], b[3][NT];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const u32x4*>(L + (t0 + i < n ? t0 + i : n - 1) * F + f);
#pragma unroll
    for (int h = 0; h < 3; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        b[h][t] = *reinterpret_cast<const u32x4*>(St + (h * 16 * NT + t * 16 + li) * n_pad + t0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t0 + i >= n) x[i] = u32x4{0u, 0u, 0u, 0u};
      if (kDrop) x[i] = drop8(x[i], key, static_cast<uint64_t>((t0 + i) * F + f), d.thr);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4 lo, hi;   // features 2 c and 2 c + 1: tokens 0 .. 7
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(x[2 * i + 1][c], x[2 * i][c], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(x[2 * i + 1][c], x[2 * i][c], 0x07060302u);
      }
#pragma unroll
      for (int h = 0; h < 3; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[2 * c][t] = mfma16(lo, b[h][t], acc[2 * c][t]);
          acc[2 * c + 1][t] = mfma16(hi, b[h][t], acc[2 * c + 1][t]);
        }
    }
  }
  // waves 2 and 3 park their sums, 0 and 1 add them; then 1 parks and 0 adds
  auto at = [&](int j, int t, int v) { return ((j * NT + t) * 4 + v) * 64 + lane; };
  if (w >= 2)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[w - 2][at(j, t, v)] = acc[j][t][v];
  __syncthreads();
  if (w < 2)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][t][v] += part[w][at(j, t, v)];
  __syncthreads();
  if (w == 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[0][at(j, t, v)] = acc[j][t][v];
  __syncthreads();
  if (w != 0) return;
  float* o = out + static_cast<int64_t>(q) * F * (16 * NT);
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t i = group * 128 + 8 * (4 * lg + v) + j;
        if (i < F) o[i * (16 * NT) + t * 16 + li] = acc[j][t][v] + part[0][at(j, t, v)];
      }
}

__global__ __launch_bounds__(kThreads) void grad_sum_kernel(const float* __restrict__ partials, int64_t F, int64_t nf,
                                                            int r, int rp, int ts, float coef, int rank_major,
                                                            float* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= nf * r) return;
  const int64_t f = rank_major ? i % nf : i / r, p = rank_major ? i / nf : i % r;
  float x = 0.f;
  for (int q = 0; q < ts; ++q) x += partials[(q * F + f) * rp + p];
  out[i] = coef * x;
}

unsigned blocks_for(int64_t threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

}  // namespace

hipError_t launch_adapter_operands(const AdapterOperands& a, hipStream_t s) {
  const int64_t n = a.rp * ((a.Ab ? a.cols : 0) + (a.Bt ? a.rows_pad : 0)) +
                    a.ld * ((a.At ? a.cols : 0) + (a.Bb ? a.rows : 0));
  LQ_LAUNCH("adapter_operands", adapter_operands_kernel, dim3(blocks_for(n)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

int down_splits(int64_t n, int64_t K) {
  const int64_t groups = n > 64 ? (n + 63) / 64 : 1;
  int64_t ks = 512 / groups;
  if (ks > K / 32 / 8) ks = K / 32 / 8;
  return static_cast<int>(ks < 1 ? 1 : (ks > 16 ? 16 : ks));
}

hipError_t launch_down(const __bf16* X, int64_t n, int64_t K, const __bf16* Mb, int rp, int ks, const DropArg& drop,
                       float* partials, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((n + 63) / 64 * ks));
#define LQ_DOWN(NT)                                                                                                    \
  do {                                                                                                                 \
    if (drop.thr != 0)                                                                                                 \
      LQ_LAUNCH("adapter_down", (down_kernel<NT, true>), grid, dim3(kThreads), 0, s, X, n, K, Mb, ks, drop, partials); \
    else                                                                                                               \
      LQ_LAUNCH("adapter_down", (down_kernel<NT, false>), grid, dim3(kThreads), 0, s, X, n, K, Mb, ks, drop, partials); \
  } while (0)
  switch (rp / 16) {
    case 1: LQ_DOWN(1); break;
    case 2: LQ_DOWN(2); break;
    case 3: LQ_DOWN(3); break;
    default: LQ_DOWN(4); break;
  }
#undef LQ_DOWN
  return hipGetLastError();
}

hipError_t launch_down_sum(const float* partials, int64_t n, int r, int rp, int ks, float gain, __bf16* S, __bf16* St,
                           int64_t n_pad, hipStream_t s) {
  LQ_LAUNCH("adapter_down_sum", down_sum_kernel, dim3(blocks_for(n_pad * rp)), dim3(kThreads), 0, s, partials, n, r, rp,
            ks, gain, adapter_ld(rp), S, St, n_pad);
  return hipGetLastError();
}

int grad_splits(int64_t n, int64_t F) {
  const int64_t groups = F > 128 ? (F + 127) / 128 : 1;
  int64_t ts = 512 / groups;
  const int64_t most = (n + 127) / 128;   // at least 128 tokens, one step of each wave
  if (ts > most) ts = most;
  return static_cast<int>(ts < 1 ? 1 : (ts > 16 ? 16 : ts));
}

hipError_t launch_grad(const __bf16* L, int64_t n, int64_t F, const __bf16* St, int rp, int64_t n_pad, int ts,
                       const DropArg& drop, float* partials, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((F + 127) / 128 * ts));
#define LQ_GRAD(NT)                                                                                                     \
  do {                                                                                                                  \
    if (drop.thr != 0)                                                                                                  \
      LQ_LAUNCH("adapter_grad", (grad_kernel<NT, true>), grid, dim3(kThreads), 0, s, L, n, F, St, n_pad, ts, drop, partials); \
    else                                                                                                                \
      LQ_LAUNCH("adapter_grad", (grad_kernel<NT, false>), grid, dim3(kThreads), 0, s, L, n, F, St, n_pad, ts, drop, partials); \
  } while (0)
  switch (rp / 16) {
    case 1: LQ_GRAD(1); break;
    case 2: LQ_GRAD(2); break;
    case 3: LQ_GRAD(3); break;
    default: LQ_GRAD(4); break;
  }
#undef LQ_GRAD
  return hipGetLastError();
}

hipError_t launch_grad_sum(const float* partials, int64_t F, int64_t nf, int r, int rp, int ts, float coef,
                           bool rank_major, float* out, hipStream_t s) {
  LQ_LAUNCH("adapter_grad_sum", grad_sum_kernel, dim3(blocks_for(nf * r)), dim3(kThreads), 0, s, partials, F, nf, r, rp,
            ts, coef, rank_major ? 1 : 0, out);
  return hipGetLastError();
}

namespace {
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

hipError_t launch_base_bf16(const Base4& b, int64_t rows, int64_t cols, __bf16* out, hipStream_t s) {
  const dim3 grid(blocks_for(rows * cols / 8));
  const Levels lv = base_levels(b);
  LQ_LAUNCH("base_bf16", (base_bf16_kernel<NfSource>), grid, dim3(kThreads), 0, s,
            (NfSource{b.packed, b.absmax, b.qabsmax, b.dq_scale}), lv, rows, cols, out);
  return hipGetLastError();
}

hipError_t launch_base_bf16_t(const Base4& b, int64_t rows, int64_t cols, int64_t rows_pad, __bf16* out,
                              hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((rows_pad / 64) * ((cols + 63) / 64)));
  const Levels lv = base_levels(b);
  if (b.mx != nullptr)
    LQ_LAUNCH("base_bf16_t", (base_bf16_t_kernel<MxSource>), grid, dim3(kThreads), 0, s, (MxSource{b.packed, b.mx}), lv,
              rows, cols, rows_pad, out);
  else
    LQ_LAUNCH("base_bf16_t", (base_bf16_t_kernel<NfSource>), grid, dim3(kThreads), 0, s,
              (NfSource{b.packed, b.absmax, b.qabsmax, b.dq_scale}), lv, rows, cols, rows_pad, out);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const __bf16* src, int64_t n, int64_t cols, int64_t ld, __bf16* dst, hipStream_t s) {
  LQ_LAUNCH("pad_rows", pad_rows_kernel, dim3(blocks_for(n * ld / 8)), dim3(kThreads), 0, s, src, n, cols, ld, dst);
  return hipGetLastError();
}

}  // namespace loftq
