// C-ABI entry points of the adapted layer's training and serving path (dropout, MXFP4, the
// training forward, the gradient): argument validation, workspace layout, then launches.
#include "entry.h"
#include "layer.h"

using namespace loftq;

namespace {

i64 pad_to(i64 n, i64 m) { return (n + m - 1) / m * m; }

// The pieces of a call's workspace.  Each is as large as any call of up to n tokens and of
// rank up to r needs it, so that the workspace of a long prompt serves a shorter one.
struct ForwardSpace {
  __bf16* W;        // NormalFloat base: bf16(deq)
  uint8_t* xq;      // MXFP4 base: the activations' codes and scales
  uint8_t* xs;
  __bf16 *Ab, *Bb, *S;
  float* partials;   // of X A^T
  float* T;          // of X A^T for the few-token product
  float* joins;      // of the product's K ranges
  int ks;
  size_t bytes;
};

ForwardSpace forward_space(void* ws, i64 n, i64 rows, i64 cols, int r, bool mx) {
  Arena a{static_cast<char*>(ws)};
  ForwardSpace f{};
  if (mx && r > 0) {
    const i64 few = n < kFewTokens ? n : kFewTokens;
    f.T = a.take<float>(lora_down_splits(few, cols, r) * few * r);   // one number of ranges up to 16 tokens
  }
  if (mx) {
    f.xq = a.take<uint8_t>(n * mx_steps(cols) * (kMxStep / 2));
    f.xs = a.take<uint8_t>(n * mx_steps(cols) * 8);
  } else {
    f.W = a.take<__bf16>(rows * cols);
  }
  if (r > 0) {
    const int rp = rank_pad(r);
    f.ks = down_splits(n, cols);
    f.Ab = a.take<__bf16>(rp * cols);
    f.Bb = a.take<__bf16>(rows * adapter_ld(rp));
    f.S = a.take<__bf16>(n * adapter_ld(rp));
    f.partials = a.take<float>(down_rows_bound(n, cols) * rp);
  }
  const int steps = static_cast<int>(mx ? mx_steps(cols) : cols / 64);
  f.joins = a.take<float>(tile_product_partial_bound(n, rows, steps) / 4);
  f.bytes = a.used;
  return f;
}

struct BackwardSpace {
  __bf16 *G, *Wt, *Ab, *At, *Bt, *Ht, *Pt, *Ps;
  float *down_p, *down_h, *grad_b, *grad_a;   // partial sums of the thin products
  float* joins;                               // of the product's K ranges
  int ks_p, ks_h, ts;
  size_t bytes;
};

BackwardSpace backward_space(void* ws, i64 n, i64 rows, i64 cols, int r) {
  Arena a{static_cast<char*>(ws)};
  BackwardSpace f{};
  const i64 rows_pad = pad_to(rows, 64), n_pad = pad_to(n, 32);
  const int rp = rank_pad(r);
  if (rows_pad != rows) f.G = a.take<__bf16>(n * rows_pad);
  f.Wt = a.take<__bf16>(cols * rows_pad);
  if (r > 0) {
    f.ks_h = down_splits(n, cols);
    f.ks_p = down_splits(n, rows_pad);
    f.ts = grad_splits(n, rows_pad, cols);
    f.Ab = a.take<__bf16>(rp * cols);
    f.At = a.take<__bf16>(cols * adapter_ld(rp));
    f.Bt = a.take<__bf16>(rp * rows_pad);
    f.Ht = a.take<__bf16>(3 * rp * n_pad);
    f.Pt = a.take<__bf16>(3 * rp * n_pad);
    f.Ps = a.take<__bf16>(n * adapter_ld(rp));
    f.down_p = a.take<float>(down_rows_bound(n, rows_pad) * rp);
    f.down_h = a.take<float>(down_rows_bound(n, cols) * rp);
    f.grad_b = a.take<float>(f.ts > 1 ? f.ts * rows_pad * rp : 0);
    f.grad_a = a.take<float>(f.ts > 1 ? f.ts * cols * rp : 0);
  }
  f.joins = a.take<float>(tile_product_partial_bound(n, cols, static_cast<int>(rows_pad / 64)) / 4);
  f.bytes = a.used;
  return f;
}

// Every launch of a call stays below 2^32 work-items, and so do the element counts that
// their 32-bit thread numbers run over.
bool layer_shape_ok(i64 n, i64 rows, i64 cols, int r) {
  const i64 limit = (i64(1) << 32) - 4096, rp = rank_pad(r), rows_pad = pad_to(rows, 64);
  if (!tile_product_shape_ok(n, rows, cols) || !tile_product_shape_ok(n, cols, 0)) return false;
  const i64 base = rows_pad * (cols / 8 + 16), codes = n * mx_steps(cols) * 32, pad = n * (rows_pad / 8);
  const i64 operands = (rp + adapter_ld(static_cast<int>(rp))) * (cols + rows_pad);
  return (base > codes ? base : codes) + pad + operands < limit && pad_to(n, 64) * 128 < limit && rows < limit / 64;
}

// Both factors or none; one of no elements may have no address.
bool factors_ok(const float* B, const float* A, i64 rows, i64 cols) {
  return rows == 0 || cols == 0 || (B == nullptr) == (A == nullptr);
}

// What the training calls share: sizes, the base, the adapter, the dropout.
loftq_status_t check_layer(i64 n, i64 rows, i64 cols, const Base4& b, bool mx, const float* B, const float* A, int r,
                           float alpha, const loftq_dropout_t* drop) {
  if (!shape_ok(rows, cols) || n < 0 || n >= (i64(1) << 31)) return LOFTQ_ERR_INVALID_ARG;
  if (!mx) {
    if (b.bits != 2 && b.bits != 3 && b.bits != 4) return LOFTQ_ERR_UNSUPPORTED;
    if (!nf_tables(b.bits).valid) return LOFTQ_ERR_UNSUPPORTED;
    if ((b.qabsmax == nullptr) != (b.dq_scale == nullptr)) return LOFTQ_ERR_INVALID_ARG;
  }
  if (!factors_ok(B, A, rows, cols)) return LOFTQ_ERR_INVALID_ARG;
  if (B != nullptr && r < 1) return LOFTQ_ERR_INVALID_ARG;
  if (!std::isfinite(alpha) || !drop_ok(drop) || !std::isfinite(alpha * drop_arg(drop).scale)) return LOFTQ_ERR_INVALID_ARG;
  return LOFTQ_OK;
}

loftq_status_t check_layer_buffers(i64 n, i64 rows, i64 cols, const Base4& b, bool mx, const float* B, const float* A,
                                   int r) {
  if (cols == 0 || cols % (mx ? kMxBlock : 64) != 0 || (B != nullptr && r > 64)) return LOFTQ_ERR_UNSUPPORTED;
  if (!layer_shape_ok(n, rows, cols, B ? r : 0)) return LOFTQ_ERR_UNSUPPORTED;
  if (!b.packed || !aligned16(b.packed)) return LOFTQ_ERR_INVALID_ARG;
  if (mx) {
    if (!b.mx || !aligned16(b.mx)) return LOFTQ_ERR_INVALID_ARG;
  } else if (b.qabsmax != nullptr) {
    if (!aligned16(b.qabsmax) || !aligned16(b.dq_scale)) return LOFTQ_ERR_INVALID_ARG;
  } else if (!b.absmax || !aligned16(b.absmax)) {
    return LOFTQ_ERR_INVALID_ARG;
  }
  if (B && (!aligned16(B) || !aligned16(A))) return LOFTQ_ERR_INVALID_ARG;
  return LOFTQ_OK;
}

loftq_status_t layer_forward(const void* X, i64 n, i64 rows, i64 cols, const Base4& base, bool mx, const float* B,
                             const float* A, int r, float alpha, const loftq_dropout_t* drop, void* Y,
                             loftq_dtype_t ydt, void* ws, size_t ws_bytes, hipStream_t s) {
  loftq_status_t st = check_layer(n, rows, cols, base, mx, B, A, r, alpha, drop);
  if (st != LOFTQ_OK) return st;
  if (!dtype_ok(ydt)) return LOFTQ_ERR_INVALID_ARG;
  if (n == 0 || rows == 0) return LOFTQ_OK;   // nothing to write
  st = check_layer_buffers(n, rows, cols, base, mx, B, A, r);
  if (st != LOFTQ_OK) return st;
  if (!X || !Y || !ws || !aligned16(X) || !aligned16(Y) || !aligned16(ws)) return LOFTQ_ERR_INVALID_ARG;
  if (B == nullptr) r = 0;
  const ForwardSpace f = forward_space(ws, n, rows, cols, r, mx);
  if (ws_bytes < f.bytes) return LOFTQ_ERR_WORKSPACE;
  const __bf16* Xb = static_cast<const __bf16*>(X);
  const DropArg d = drop_arg(drop);
  if (mx && (r == 0 || d.thr == 0) && token_product_pays(n, rows, cols, r)) {   // dropout is the tiled path's
    if (r > 0) LQ_TRY(launch_lora_down(Xb, n, cols, A, r, f.T, s));
    return from_hip(launch_token_product(TokenProduct{Xb, base.packed, base.mx, f.T, B, n, rows, cols,
                                                      r > 0 ? lora_down_splits(n, cols, r) : 0, r, alpha, Y, ydt}, s));
  }
  const int rp = rank_pad(r);
  PrepareArgs p{};
  p.a = AdapterOperands{A, B, r, rp, rows, cols, rows, f.Ab, nullptr, f.Bb, nullptr, adapter_ld(rp)};
  p.n = n;
  TileProduct t{};
  t.M = n;
  t.N = rows;
  if (mx) {
    p.x = Xb;
    p.xq = f.xq;
    p.xs = f.xs;
    p.steps = mx_steps(cols);
    t.W = base.packed;
    t.X = f.xq;
    t.steps = static_cast<int>(p.steps);
    t.ldw = t.ldx = t.steps * i64(kMxStep / 2);
    t.wscale = base.mx;
    t.xscale = f.xs;
  } else {
    p.base = f.W;
    t.W = f.W;
    t.X = Xb;
    t.steps = static_cast<int>(cols / 64);
    t.ldw = t.ldx = cols * 2;
  }
  LQ_TRY(launch_prepare(p, base, mx ? kBaseCodesOfX : kBaseAsItLies, s));
  if (r > 0) {
    LQ_TRY(launch_down(DownJobs{{{Xb, f.Ab, f.partials, cols, f.ks, 0, d}, {}}}, n, rp, s));
    LQ_TRY(launch_down_sum(DownSumJobs{{{f.partials, f.ks, alpha * d.scale, f.S, nullptr, 0}, {}}}, n, r, rp, s));
    t.V = f.Bb;
    t.S = f.S;
    t.adapter_steps = adapter_ld(rp) / 64;
  }
  t.out = Y;
  t.odt = ydt;
  return from_hip(launch_tile_product(t, mx, f.joins, s));
}

loftq_status_t layer_backward(const void* dY, const void* X, i64 n, i64 rows, i64 cols, const Base4& base, bool mx,
                              const float* B, const float* A, int r, float alpha, const loftq_dropout_t* drop,
                              void* dX, loftq_dtype_t xdt, float* dB, float* dA, void* ws, size_t ws_bytes,
                              hipStream_t s) {
  loftq_status_t st = check_layer(n, rows, cols, base, mx, B, A, r, alpha, drop);
  if (st != LOFTQ_OK) return st;
  if (dX && !dtype_ok(xdt)) return LOFTQ_ERR_INVALID_ARG;
  if ((dB == nullptr) != (dA == nullptr) || (dB && !B)) return LOFTQ_ERR_INVALID_ARG;
  if (!dX && !dB && n > 0) return LOFTQ_ERR_INVALID_ARG;   // without tokens dX has no elements and may have no address
  if (rows == 0 || rows >= i64(1) << 22) return LOFTQ_ERR_UNSUPPORTED;   // rows are the product's K
  st = check_layer_buffers(n, rows, cols, base, mx, B, A, r);
  if (st != LOFTQ_OK) return st;
  if ((dX && !aligned16(dX)) || (dB && (!aligned16(dB) || !aligned16(dA)))) return LOFTQ_ERR_INVALID_ARG;
  if (B == nullptr) r = 0;
  const int rp = rank_pad(r);
  if (n == 0) {   // sums over no tokens: no partials, so zeros
    if (dB) LQ_TRY(launch_grad_sum(GradJobs{{{nullptr, nullptr, nullptr, dB, rows, rows}, {nullptr, nullptr, nullptr, dA, cols, cols}}}, r, rp, s));
    return LOFTQ_OK;
  }
  if (!dY || !ws || !aligned16(dY) || !aligned16(ws)) return LOFTQ_ERR_INVALID_ARG;
  if (dB && (!X || !aligned16(X))) return LOFTQ_ERR_INVALID_ARG;
  const BackwardSpace f = backward_space(ws, n, rows, cols, r);
  if (ws_bytes < f.bytes) return LOFTQ_ERR_WORKSPACE;
  const DropArg d = drop_arg(drop), none = drop_arg(nullptr);
  const float gain = alpha * d.scale;
  const i64 rows_pad = pad_to(rows, 64);
  const __bf16* G = static_cast<const __bf16*>(dY);
  const __bf16* Xb = static_cast<const __bf16*>(X);
  PrepareArgs p{};
  p.a = AdapterOperands{A, B, r, rp, rows, cols, rows_pad, dB ? f.Ab : nullptr, dX ? f.At : nullptr, nullptr, f.Bt,
                        adapter_ld(rp)};
  p.base = f.Wt;
  p.n = n;
  p.x = G;
  p.padded = f.G;
  LQ_TRY(launch_prepare(p, base, dX ? kBaseTransposed : kBaseNone, s));
  if (f.G != nullptr) G = f.G;
  if (r > 0) {
    // P = G B for dX and dA, H = keep(X) A^T for dB
    DownJobs down{{{G, f.Bt, f.down_p, rows_pad, f.ks_p, 0, none}, {}}};
    DownSumJobs sum{{{f.down_p, f.ks_p, gain, dX ? f.Ps : nullptr, dB ? f.Pt : nullptr, 0}, {}}};
    if (dB) {
      down.job[1] = DownJob{Xb, f.Ab, f.down_h, cols, f.ks_h, 0, d};
      sum.job[1] = DownSumJob{f.down_h, f.ks_h, gain, nullptr, f.Ht, 0};
    }
    LQ_TRY(launch_down(down, n, rp, s));
    LQ_TRY(launch_down_sum(sum, n, r, rp, s));
    if (dB) {
      const GradJobs grad{{{G, f.Ht, f.grad_b, dB, rows_pad, rows, f.ts, gain, 0, none},
                           {Xb, f.Pt, f.grad_a, dA, cols, cols, f.ts, gain, 0, d}}};
      LQ_TRY(launch_grad(grad, n, r, rp, s));
      if (f.ts > 1) LQ_TRY(launch_grad_sum(grad, r, rp, s));
    }
  }
  if (!dX) return LOFTQ_OK;
  TileProduct t{};
  t.W = f.Wt;
  t.X = G;
  t.ldw = t.ldx = rows_pad * 2;
  t.M = n;
  t.N = cols;
  t.steps = static_cast<int>(rows_pad / 64);
  if (r > 0) {
    t.V = f.At;
    t.S = f.Ps;
    t.adapter_steps = adapter_ld(rp) / 64;
    t.drop = d;
  }
  t.out = dX;
  t.odt = xdt;
  return from_hip(launch_tile_product(t, false, f.joins, s));
}

Base4 nf_base(const uint8_t* packed, const float* absmax, const int8_t* qabsmax, const float* dq_scale, int32_t bits) {
  Base4 b;
  b.packed = packed;
  b.absmax = absmax;
  b.qabsmax = qabsmax;
  b.dq_scale = dq_scale;
  b.bits = bits;
  return b;
}

Base4 mx_base(const uint8_t* packed, const uint8_t* scales) {
  Base4 b;
  b.packed = packed;
  b.mx = scales;
  return b;
}

// 0 where a workspace query's sizes are none that the call would take
bool query_ok(i64 n, i64 rows, i64 cols, int32_t r) {
  return shape_ok(rows, cols) && n >= 0 && n < (i64(1) << 31) && r >= 0 && r <= 64 && layer_shape_ok(n, rows, cols, r);
}

}  // namespace

extern "C" {

loftq_status_t loftq_dropout(const void* X, loftq_dtype_t dt, int64_t n, const loftq_dropout_t* drop, void* Y,
                             void* stream) {
  if (!dtype_ok(dt) || n < 0 || drop == nullptr || !drop_ok(drop)) return LOFTQ_ERR_INVALID_ARG;
  if (n == 0) return LOFTQ_OK;
  if (!X || !Y || !aligned16(X) || !aligned16(Y)) return LOFTQ_ERR_INVALID_ARG;
  return from_hip(launch_dropout(X, dt, n, drop_arg(drop), Y, static_cast<hipStream_t>(stream)));
}

size_t loftq_mxfp4_packed_bytes(int64_t rows, int64_t cols) {
  return shape_ok(rows, cols) ? static_cast<size_t>(rows * mx_steps(cols) * (kMxStep / 2)) : 0;
}

size_t loftq_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
  return shape_ok(rows, cols) ? static_cast<size_t>(rows * mx_steps(cols) * (kMxStep / kMxBlock)) : 0;
}

loftq_status_t loftq_mxfp4_quantize(const void* W, loftq_dtype_t wdt, int64_t rows, int64_t cols, const float* B,
                                    const float* A, int32_t r, uint8_t* packed, uint8_t* scales, void* stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(wdt)) return LOFTQ_ERR_INVALID_ARG;
  if (!factors_ok(B, A, rows, cols)) return LOFTQ_ERR_INVALID_ARG;
  if (B != nullptr && (r < 1 || r > 4096)) return LOFTQ_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return LOFTQ_OK;
  if (!mx_shape_ok(rows, cols)) return LOFTQ_ERR_UNSUPPORTED;
  if (!W || !packed || !scales) return LOFTQ_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(packed) || !aligned16(scales)) return LOFTQ_ERR_INVALID_ARG;
  if (B && (!aligned16(B) || !aligned16(A))) return LOFTQ_ERR_INVALID_ARG;
  return from_hip(launch_mx_quantize(W, wdt, rows, cols, B, A, B ? r : 0, packed, scales,
                                     static_cast<hipStream_t>(stream)));
}

loftq_status_t loftq_mxfp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t cols,
                                      const void* W, loftq_dtype_t wdt, void* out, loftq_dtype_t odt, void* stream) {
  if (!shape_ok(rows, cols) || !dtype_ok(odt) || (W && !dtype_ok(wdt))) return LOFTQ_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return LOFTQ_OK;
  if (!mx_shape_ok(rows, cols)) return LOFTQ_ERR_UNSUPPORTED;
  if (!packed || !scales || !out) return LOFTQ_ERR_INVALID_ARG;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(out) || (W && !aligned16(W))) return LOFTQ_ERR_INVALID_ARG;
  return from_hip(launch_mx_dequantize(packed, scales, rows, cols, W, wdt, out, odt, static_cast<hipStream_t>(stream)));
}

loftq_status_t loftq_qlora_forward_dropout(const void* X, int64_t n_tok, int64_t rows, int64_t cols,
                                           const uint8_t* packed, const float* absmax, const int8_t* qabsmax,
                                           const float* dq_scale, int32_t bits, const float* B, const float* A,
                                           int32_t r, float alpha, const loftq_dropout_t* drop, void* Y,
                                           loftq_dtype_t ydt, void* ws, size_t ws_bytes, void* stream) {
  return layer_forward(X, n_tok, rows, cols, nf_base(packed, absmax, qabsmax, dq_scale, bits), false, B, A, r, alpha,
                       drop, Y, ydt, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

loftq_status_t loftq_mxfp4_forward(const void* X, int64_t n_tok, int64_t rows, int64_t cols, const uint8_t* packed,
                                   const uint8_t* scales, const float* B, const float* A, int32_t r, float alpha,
                                   const loftq_dropout_t* drop, void* Y, loftq_dtype_t ydt, void* ws, size_t ws_bytes,
                                   void* stream) {
  return layer_forward(X, n_tok, rows, cols, mx_base(packed, scales), true, B, A, r, alpha, drop, Y, ydt, ws, ws_bytes,
                       static_cast<hipStream_t>(stream));
}

loftq_status_t loftq_qlora_backward(const void* dY, const void* X, int64_t n_tok, int64_t rows, int64_t cols,
                                    const uint8_t* packed, const float* absmax, const int8_t* qabsmax,
                                    const float* dq_scale, int32_t bits, const float* B, const float* A, int32_t r,
                                    float alpha, const loftq_dropout_t* drop, void* dX, loftq_dtype_t xdt, float* dB,
                                    float* dA, void* ws, size_t ws_bytes, void* stream) {
  return layer_backward(dY, X, n_tok, rows, cols, nf_base(packed, absmax, qabsmax, dq_scale, bits), false, B, A, r,
                        alpha, drop, dX, xdt, dB, dA, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

loftq_status_t loftq_mxfp4_backward(const void* dY, const void* X, int64_t n_tok, int64_t rows, int64_t cols,
                                    const uint8_t* packed, const uint8_t* scales, const float* B, const float* A,
                                    int32_t r, float alpha, const loftq_dropout_t* drop, void* dX, loftq_dtype_t xdt,
                                    float* dB, float* dA, void* ws, size_t ws_bytes, void* stream) {
  return layer_backward(dY, X, n_tok, rows, cols, mx_base(packed, scales), true, B, A, r, alpha, drop, dX, xdt, dB, dA,
                        ws, ws_bytes, static_cast<hipStream_t>(stream));
}

size_t loftq_qlora_forward_dropout_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t r) {
  return query_ok(n_tok, rows, cols, r) ? forward_space(nullptr, n_tok, rows, cols, r, false).bytes : 0;
}

size_t loftq_mxfp4_forward_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t r) {
  return query_ok(n_tok, rows, cols, r) ? forward_space(nullptr, n_tok, rows, cols, r, true).bytes : 0;
}

size_t loftq_qlora_backward_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t r) {
  return query_ok(n_tok, rows, cols, r) ? backward_space(nullptr, n_tok, rows, cols, r).bytes : 0;
}

size_t loftq_mxfp4_backward_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t r) {
  return loftq_qlora_backward_workspace_bytes(n_tok, rows, cols, r);
}

}  // extern "C"
