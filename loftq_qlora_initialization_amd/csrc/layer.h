// The adapted layer's training and serving path: what its translation units share.
#pragma once

#include "dropout.h"
#include "internal.h"
#include "mxfp4.h"

namespace loftq {

// A frozen 4-bit weight (rows x cols): NormalFloat codes with absmax or double-quantized
// scales, or MXFP4 codes with their scales (then `mx` is set).
struct Base4 {
  const uint8_t* packed = nullptr;
  const float* absmax = nullptr;
  const int8_t* qabsmax = nullptr;
  const float* dq_scale = nullptr;
  const uint8_t* mx = nullptr;
  int bits = 4;
};

// One tiled product C[m][n] = sum_k X[m][k] W[n][k] + keep(m, n) sum_p S[m][p] V[n][p]
// (tokens m, features n), all operands with their K in whole 128-byte steps.
struct TileProduct {
  const void* W;              // N rows of `steps` 128-byte steps, ldw bytes apart
  const void* X;              // M rows, ldx bytes apart
  int64_t ldw, ldx;
  const uint8_t* wscale;      // MXFP4: 8 bytes per row and step, [steps][N][8] and [steps][M][8]
  const uint8_t* xscale;
  int64_t M, N;
  int steps;
  const __bf16* V;            // [N][adapter_steps 64]: the factor, three times over
  const __bf16* S;            // [M][adapter_steps 64]: three bf16 pieces of each fp32 value
  int adapter_steps;          // 0: no second term
  DropArg drop;               // thr != 0: the second term is kept where the mask keeps (m N + n)
  void* out;
  loftq_dtype_t odt;
  int splits;                 // K ranges, set by the launcher
};

// How a product is divided: a tile shape and K ranges.
struct TilePlan {
  int shape, splits;
};
TilePlan plan_tile_product(int64_t M, int64_t N, int steps, int adapter_steps, bool mx);
// at least the bytes of the K ranges' partial outputs in every plan for up to M tokens, with an adapter or without
size_t tile_product_partial_bound(int64_t M, int64_t N, int steps);
hipError_t launch_tile_product(TileProduct t, bool mx, float* partials, hipStream_t s);
bool tile_product_shape_ok(int64_t M, int64_t N, int64_t K);

// The MXFP4 product for M <= kFewTokens tokens, from X itself (token_product.hip), and whether it
// is faster than the tiled one.
constexpr int64_t kFewTokens = 16;
bool token_product_pays(int64_t M, int64_t N, int64_t K, int r);
struct TokenProduct {
  const __bf16* X;            // M x K, K % 32 == 0
  const uint8_t* W;
  const uint8_t* wscale;
  const float* T;             // [ks][M][r] partials of X A^T
  const float* B;             // N x r
  int64_t M, N, K;
  int ks, r;                  // r = 0: no adapter
  float alpha;
  void* out;
  loftq_dtype_t odt;
};
hipError_t launch_token_product(const TokenProduct& t, hipStream_t s);

// ---- adapter and base operands (adapter_kernels.hip) ----
struct AdapterOperands {
  const float* A;   // r x cols
  const float* B;   // rows x r
  int r, rp;
  int64_t rows, cols, rows_pad;
  __bf16* Ab;       // [rp][cols] or null
  __bf16* At;       // [cols][ld] or null: the rank three times over, zeros behind it
  __bf16* Bb;       // [rows][ld] or null, likewise
  __bf16* Bt;       // [rp][rows_pad] or null
  int ld;           // adapter_ld(rp)
};
// elements of a row of the adapter's operands in the tiled product: three times the padded rank, in whole steps
inline int adapter_ld(int rp) { return (3 * rp + 63) / 64 * 64; }

// What a call's products read: the base's bf16 operand (as it lies, or transposed with zeros
// past `rows`), or over MXFP4 the codes of X; the adapter's operands; dY with padded rows.
enum PrepareBase { kBaseNone, kBaseAsItLies, kBaseTransposed, kBaseCodesOfX };
struct PrepareArgs {
  AdapterOperands a;       // r = 0: no adapter (rows, cols, rows_pad still hold)
  __bf16* base;
  int64_t n;               // tokens
  const __bf16* x;         // X for its codes, dY for its padding
  uint8_t *xq, *xs;        // X's codes and scales
  int64_t steps;           // mx_steps(cols)
  __bf16* padded;          // dY in rows of rows_pad, or null
  unsigned base_wgs, operand_wgs;   // set by the launcher
};
hipError_t launch_prepare(PrepareArgs p, const Base4& b, PrepareBase kind, hipStream_t s);

// P = keep(X) M^T as K-split partials [ks][n][rp] (X null: no such job); then the sum in split
// order as three bf16 pieces, of gain P token-major in S [n][adapter_ld(rp)], of P rank-major
// in St [3][rp][n_pad] (either may be null; n_pad = n in whole 32s).
struct DownJob {
  const __bf16 *X, *M;
  float* out;
  int64_t K;
  int ks;
  unsigned wgs;            // set by the launcher
  DropArg drop;
};
struct DownJobs {
  DownJob job[2];
};
struct DownSumJob {
  const float* partials;
  int ks;
  float gain;
  __bf16 *S, *St;
  unsigned wgs;            // set by the launcher
};
struct DownSumJobs {
  DownSumJob job[2];
};
int down_splits(int64_t n, int64_t K);
int64_t down_rows_bound(int64_t n, int64_t K);   // at least down_splits(m, K) m for every m <= n
hipError_t launch_down(DownJobs jobs, int64_t n, int rp, hipStream_t s);
hipError_t launch_down_sum(DownSumJobs jobs, int64_t n, int r, int rp, hipStream_t s);

// out[i][p] = coef sum_t keep(L)[t][i] (fp32 value of St)[p][t] for i < nf, p < r: job 0 (dB)
// feature-major over dY, job 1 (dA) rank-major over X with its mask.  L has F >= nf columns.
// Over ts > 1 token ranges the sums go to `partials` ([ts][F][rp], [ts][rp][F]) and
// launch_grad_sum adds them; over one they are written to `out` at once.
struct GradJob {
  const __bf16 *L, *St;
  float *partials, *out;
  int64_t F, nf;
  int ts;
  float coef;
  unsigned wgs;            // set by the launcher
  DropArg drop;
};
struct GradJobs {
  GradJob job[2];
};
int grad_splits(int64_t n, int64_t rows_pad, int64_t cols);
hipError_t launch_grad(GradJobs jobs, int64_t n, int r, int rp, hipStream_t s);
hipError_t launch_grad_sum(const GradJobs& jobs, int r, int rp, hipStream_t s);

// ---- MXFP4 (mxfp4_kernels.hip) ----
bool mx_shape_ok(int64_t rows, int64_t cols);
hipError_t launch_mx_quantize(const void* W, loftq_dtype_t wdt, int64_t rows, int64_t cols, const float* B,
                              const float* A, int r, uint8_t* packed, uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t cols,
                                const void* W, loftq_dtype_t wdt, void* out, loftq_dtype_t odt, hipStream_t s);

hipError_t launch_dropout(const void* X, loftq_dtype_t dt, int64_t n, const DropArg& d, void* Y, hipStream_t s);

}  // namespace loftq
