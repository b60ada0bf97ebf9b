// The adapted layer over an MXFP4 base for a few tokens (serving): bound by reading the weight,
// and by the launches before it, so the tokens' codes are formed where they are multiplied.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 on FP4: lane L supplies row L%16, k = 32 (L/16) .. + 31,
// one MXFP4 block with its scale byte, for either operand; tokens are the first, so lane L
// receives token 4 (L/16) + v, feature L%16 in element v.
//
// A workgroup owns 16 NF features and up to 16 tokens; its waves take steps of 256 columns in
// turn (whole lines of the weight's codes).  A lane holds a whole block of a token: it finds
// the scale and the codes by itself, as mx_quantize_kernel does, so a token's result is that of
// the tiled product up to the order of its sums.  That repeats the tokens' rounding in every
// workgroup, and reads four times a feature tile's bytes for it: NF tiles share it where the
// features suffice.  The partial sums meet in LDS in wave order, then the adapter's term is
// added in fp32.
#include "layer.h"

namespace loftq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 16, kChunk = 128;

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// A block of 32 values into its codes and scale byte.
__device__ __forceinline__ i32x4 encode_block(const bf16x8 (&x)[4], uint32_t& byte) {
  uint32_t amax = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(static_cast<float>(x[q][j])) & 0x7FFFFFFFu;
      amax = b > amax ? b : amax;
    }
  byte = mx_scale_byte(amax);
  const float inv = mx_inverse_scale(byte);
  i32x4 out;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(x[q][j]) * inv;
    out[q] = static_cast<int>(mx_codes8(v));
  }
  return out;
}

template <int NF, typename O>
__global__ __launch_bounds__(kWaves * 64) void token_product_kernel(TokenProduct t) {
  __shared__ float part[kWaves / 2][NF * 256];
  __shared__ float Ts[16 * 64];         // the tokens' rows of X A^T, r <= 64
  __shared__ float Bs[NF * 16 * 64];    // bf16(B) of the workgroup's features
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, li = lane & 15, lg = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NF), M = t.M, N = t.N, K = t.K;
  const int r = t.r;
  // the epilogue's operands first, their loads beside the main loop's
  if (r > 0) {
    for (int i = tid; i < M * r; i += kWaves * 64) {
      float x = 0.f;
      for (int q = 0; q < t.ks; ++q) x += t.T[q * M * r + i];
      Ts[i] = x;
    }
    for (int i = tid; i < NF * 16 * r; i += kWaves * 64) {
      const int64_t n = n0 + i / r < N ? n0 + i / r : N - 1;
      Bs[i] = static_cast<float>(static_cast<__bf16>(t.B[n * r + i % r]));
    }
  }
  const int64_t steps = (K + kMxStep - 1) / kMxStep;
  int64_t n[NF];   // rows past the last repeat it (never stored)
#pragma unroll
  for (int f = 0; f < NF; ++f) n[f] = n0 + f * 16 + li < N ? n0 + f * 16 + li : N - 1;
  const int64_t m = li < M ? li : M - 1;
  f32x4 acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the two chunks of a step at a time: whole lines of the codes; blocks past K (K % 32 == 0)
  // load a valid address and count as zeros
  for (int64_t k0 = static_cast<int64_t>(w) * kMxStep; k0 < K; k0 += kWaves * kMxStep) {
    i32x4 wc[2][NF];
    uint32_t ws[2][NF];
    bf16x8 x[2][4];
    bool live[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = k0 + u * kChunk + 32 * lg;
      live[u] = k < K;
      const int64_t kk = live[u] ? k : 0;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        wc[u][f] = *reinterpret_cast<const i32x4*>(t.W + n[f] * steps * (kMxStep / 2) + kk / 2);
        ws[u][f] = t.wscale[(kk / kMxStep * N + n[f]) * 8 + kk % kMxStep / kMxBlock];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) x[u][q] = *reinterpret_cast<const bf16x8*>(t.X + m * K + kk + 8 * q);
    }
    __builtin_amdgcn_sched_barrier(0);   // every load of the step is in flight before the first wait
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const i32x4 zero = {0, 0, 0, 0};
      uint32_t byte;
      i32x4 xv = encode_block(x[u], byte);
      xv = live[u] ? xv : zero;
      byte = live[u] ? byte : 0u;
#pragma unroll
      for (int f = 0; f < NF; ++f)
        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(xv), widen(live[u] ? wc[u][f] : zero), acc[f], 4, 4,
                                                                  0, static_cast<int>(byte), 0,
                                                                  static_cast<int>(live[u] ? ws[u][f] : 0u));
    }
  }
  auto at = [&](int f, int v) { return (f * 4 + v) * 64 + lane; };
  if (w >= kWaves / 2)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[w - kWaves / 2][at(f, v)] = acc[f][v];
  __syncthreads();
  if (w < kWaves / 2)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[w][at(f, v)] += acc[f][v];
  __syncthreads();
  for (int e = tid; e < NF * 256; e += kWaves * 64) {
    const int ln = e & 63, v = (e >> 6) & 3, f = e >> 8;
    const int64_t mm = 4 * (ln >> 4) + v, nn = n0 + f * 16 + (ln & 15);
    if (mm >= M || nn >= N) continue;
    float y = 0.f;
#pragma unroll
    for (int q = 0; q < kWaves / 2; ++q) y += part[q][e];
    float lora = 0.f;
    for (int p = 0; p < r; ++p) lora = fmaf(Ts[mm * r + p], Bs[(f * 16 + (ln & 15)) * r + p], lora);
    if (r > 0) y = fmaf(t.alpha, lora, y);
    static_cast<O*>(t.out)[mm * N + nn] = static_cast<O>(y);
  }
}

// Feature tiles a workgroup: as many as leave each CU one.
int feature_tiles(int64_t N) { return N >= 16384 ? 4 : (N >= 8192 ? 2 : 1); }

}  // namespace

// Both sides with their launches, in a graph, weights read from memory (us, this against tiled):
//                  r = 16, 1 token   8 tokens         r = 64, 1 token   8 tokens
//   4096 x  4096   9.8  against 21.5 11.7        22.3 13.7        26.0  16.9        27.4
//  11008 x  4096   18.9         23.9 22.0        24.6 24.4        29.0  32.5        29.8
//   8192 x  8192   19.0         27.8 20.2        27.9 25.5        31.8  30.1        32.9
//  22016 x  4096   25.2         28.6 29.0        28.9 33.8        36.3  49.8        37.2
//  16384 x  8192   27.4         34.5 29.6        34.0 36.2        40.2  42.7        41.3
//  11008 x 11008   35.0         33.0 40.8        33.7 46.4        39.2  56.7        40.3
//  28672 x  8192   45.1         44.5 51.2        44.7 55.6        55.1  71.8        56.8
//     64 x 11008   15.8         20.1 19.2        20.0 25.3        23.2  30.0        24.3
//   1024 x 16384   20.5         21.3 23.8        23.1 32.2        26.3  36.4        28.1
//    128 x 65536   64.9         31.7 77.1        32.6 107         41.5  121         43.9
// Up to 2^25 weights one round of workgroups takes them all, and what counts is the length of K
// that a workgroup goes through, with the adapter's and the tokens' share of a step; past them
// the weight with its features in whole rounds, and for the adapter's end M r.
bool token_product_pays(int64_t M, int64_t N, int64_t K, int r) {
  if (M > kFewTokens) return false;
  if (N * K <= (int64_t(1) << 25)) return K * (72 + 2 * r + 5 * M) <= (int64_t(1) << 21);
  const int64_t round = 256 * 16 * feature_tiles(N), size = (N + round - 1) / round * round * K;
  return M <= 8 && size <= (int64_t(1) << 27) && M * r * size <= (int64_t(1) << 34);
}

hipError_t launch_token_product(const TokenProduct& t, hipStream_t s) {
  const int nf = feature_tiles(t.N);
  const dim3 grid(static_cast<unsigned>((t.N + 16 * nf - 1) / (16 * nf))), block(kWaves * 64);
#define LQ_TOKEN(NF, O) LQ_LAUNCH("mx_token_product", (token_product_kernel<NF, O>), grid, block, 0, s, t)
#define LQ_TOKEN_O(O)                \
  do {                               \
    if (nf == 4) LQ_TOKEN(4, O);     \
    else if (nf == 2) LQ_TOKEN(2, O); \
    else LQ_TOKEN(1, O);             \
  } while (0)
  if (t.odt == LOFTQ_BF16) LQ_TOKEN_O(__bf16);
  else LQ_TOKEN_O(float);
#undef LQ_TOKEN_O
#undef LQ_TOKEN
  return hipGetLastError();
}

}  // namespace loftq
