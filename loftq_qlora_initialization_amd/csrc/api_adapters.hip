// C-ABI entry points of many adapters beside one shared weight: argument validation, workspace
// layout, then launches.
#include "adapters.h"
#include "entry.h"

using namespace loftq;

namespace {

constexpr i64 kMostTokens = i64(1) << 25, kMostWidth = i64(1) << 22, kMostWorkgroups = i64(1) << 22;
constexpr i64 kFewAdapterTokens = 256;

i64 pad8(i64 n) { return (n + 7) / 8 * 8; }

bool plan_sizes_ok(i64 n, int slots) { return n < kMostTokens && slots <= kMostSlots; }

// Every launch of a call stays below 2^32 work-items.
bool sizes_ok(i64 n, i64 rows, i64 cols, int slots, int rank, bool backward) {
  if (!plan_sizes_ok(n, slots) || rank > 64 || rows >= kMostWidth || cols >= kMostWidth || cols == 0 || cols % 8 != 0) return false;
  if (backward && rows == 0) return false;
  const PlanLayout p = plan_layout(n, slots);
  const i64 features = backward ? cols : rows, rp = rank_pad(rank);
  // the threads that make the factors' forms
  const i64 forms = backward ? pad8(rows) / 8 * rp + 2 * cols * (rp / 8) : rows * (rp / 8);
  if ((forms + 1024) * slots >= (i64(1) << 31)) return false;
  if (p.max_tiles * ((features + 255) / 256) >= kMostWorkgroups) return false;
  if (!backward) return true;
  if (p.max_chunks * ((pad8(rows) + 127) / 128 + (cols + 127) / 128) >= 2 * kMostWorkgroups) return false;
  return n * (pad8(rows) / 8) < (i64(1) << 32) - 4096;
}

struct ForwardSpace {
  float* partials;   // of X A^T
  float* H;          // their sum
  __bf16* Bp;        // B in bf16 rows of whole 16 ranks, unless it is read as it lies
  int ks;
  size_t bytes;
};
ForwardSpace forward_space(void* ws, i64 n, i64 rows, i64 cols, int slots, int rank) {
  Arena a{static_cast<char*>(ws)};
  ForwardSpace f{};
  const int rp = rank_pad(rank);
  f.ks = adapters_down_splits(n, slots, cols, rp);
  f.partials = a.take<float>(adapters_down_floats_bound(n, slots, cols, rp));
  f.H = a.take<float>(plan_layout(n, slots).max_tiles * kTile * rp);
  f.Bp = a.take<__bf16>(used_slots(n, slots) * rows * rp);
  f.bytes = a.used;
  return f;
}

struct BackwardSpace {
  __bf16 *G, *Pt, *Ht, *Bt, *Ab, *At;
  float *down_p, *down_h, *P, *grad_b, *grad_a;
  int ks_p, ks_h;
  size_t bytes;
};
BackwardSpace backward_space(void* ws, i64 n, i64 rows, i64 cols, int slots, int rank) {
  Arena a{static_cast<char*>(ws)};
  BackwardSpace f{};
  const i64 rows8 = pad8(rows), used = used_slots(n, slots);
  const int rp = rank_pad(rank);
  const PlanLayout p = plan_layout(n, slots);
  f.ks_p = adapters_down_splits(n, slots, rows8, rp);
  f.ks_h = adapters_down_splits(n, slots, cols, rp);
  if (rows8 != rows) f.G = a.take<__bf16>(n * rows8);
  f.Bt = a.take<__bf16>(used * rows8 * rp);
  f.Ab = a.take<__bf16>(used * cols * rp);
  f.At = a.take<__bf16>(used * cols * rp);
  f.down_p = a.take<float>(adapters_down_floats_bound(n, slots, rows8, rp));
  f.down_h = a.take<float>(adapters_down_floats_bound(n, slots, cols, rp));
  f.P = a.take<float>(p.max_tiles * kTile * rp);
  f.Pt = a.take<__bf16>(3 * p.max_tiles * kTile * rp);
  f.Ht = a.take<__bf16>(3 * p.max_tiles * kTile * rp);
  f.grad_b = a.take<float>(p.max_parts * rows8 * rp);
  f.grad_a = a.take<float>(p.max_parts * cols * rp);
  f.bytes = a.used;
  return f;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes, types and numbers of a call; then, where it has work, its pool.
loftq_status_t check_call(i64 n, i64 rows, i64 cols, const loftq_adapters_t* ad, const loftq_dropout_t* drop) {
  if (!shape_ok(rows, cols) || n < 0 || n >= (i64(1) << 31) || ad == nullptr) return LOFTQ_ERR_INVALID_ARG;
  if (ad->slots < 1 || ad->rank < 1 || !dtype_ok(ad->dt) || !std::isfinite(ad->alpha) || !drop_ok(drop)) return LOFTQ_ERR_INVALID_ARG;
  return std::isfinite(ad->alpha * drop_arg(drop).scale) ? LOFTQ_OK : LOFTQ_ERR_INVALID_ARG;
}
loftq_status_t check_pool(const loftq_adapters_t* ad, const int32_t* plan, size_t plan_bytes, i64 n) {
  if (!ad->B || !ad->A || !aligned16(ad->B) || !aligned16(ad->A)) return LOFTQ_ERR_INVALID_ARG;
  if (!aligned4(ad->ranks) || !aligned4(ad->gains)) return LOFTQ_ERR_INVALID_ARG;
  if (!plan || !aligned16(plan)) return LOFTQ_ERR_INVALID_ARG;
  return plan_bytes < static_cast<size_t>(plan_layout(n, ad->slots).words) * 4 ? LOFTQ_ERR_WORKSPACE : LOFTQ_OK;
}
Pool pool_of(const loftq_adapters_t* ad, const DropArg& d) {
  return Pool{ad->B, ad->A, ad->dt, ad->slots, ad->rank, rank_pad(ad->rank), ad->ranks, ad->gains, ad->alpha * d.scale};
}

bool query_ok(i64 n, i64 rows, i64 cols, int32_t slots, int32_t rank, bool backward) {
  return shape_ok(rows, cols) && n >= 0 && n < (i64(1) << 31) && slots >= 1 && rank >= 1 &&
         sizes_ok(n, rows, cols, slots, rank, backward);
}

}  // namespace

extern "C" {

size_t loftq_adapters_plan_bytes(int64_t n_tok, int32_t slots) {
  if (n_tok < 0 || slots < 1 || !plan_sizes_ok(n_tok, slots)) return 0;
  return static_cast<size_t>(plan_layout(n_tok, slots).words) * 4;
}

loftq_status_t loftq_adapters_plan(const int32_t* slot_of, int64_t n_tok, int32_t slots, int32_t* plan, size_t plan_bytes,
                                   void* stream) {
  if (n_tok < 0 || n_tok >= (i64(1) << 31) || slots < 1) return LOFTQ_ERR_INVALID_ARG;
  if (!plan_sizes_ok(n_tok, slots)) return LOFTQ_ERR_UNSUPPORTED;
  if ((n_tok > 0 && !slot_of) || !aligned4(slot_of) || !plan || !aligned16(plan)) return LOFTQ_ERR_INVALID_ARG;
  const PlanLayout p = plan_layout(n_tok, slots);
  if (plan_bytes < static_cast<size_t>(p.words) * 4) return LOFTQ_ERR_WORKSPACE;
  return from_hip(launch_adapters_plan(slot_of, plan, p, static_cast<hipStream_t>(stream)));
}

size_t loftq_adapters_forward_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t slots, int32_t rank) {
  return query_ok(n_tok, rows, cols, slots, rank, false) && n_tok > 0 ? forward_space(nullptr, n_tok, rows, cols, slots, rank).bytes : 0;
}

loftq_status_t loftq_adapters_forward(const void* X, int64_t n_tok, int64_t rows, int64_t cols, const loftq_adapters_t* ad,
                                      const int32_t* plan, size_t plan_bytes, const loftq_dropout_t* drop, const void* Y0,
                                      void* Y, loftq_dtype_t ydt, void* ws, size_t ws_bytes, void* stream) {
  loftq_status_t st = check_call(n_tok, rows, cols, ad, drop);
  if (st != LOFTQ_OK) return st;
  if (!dtype_ok(ydt)) return LOFTQ_ERR_INVALID_ARG;
  if (n_tok == 0 || rows == 0) return LOFTQ_OK;   // nothing to write
  if (!sizes_ok(n_tok, rows, cols, ad->slots, ad->rank, false)) return LOFTQ_ERR_UNSUPPORTED;
  st = check_pool(ad, plan, plan_bytes, n_tok);
  if (st != LOFTQ_OK) return st;
  if (!X || !Y || !ws || !aligned16(X) || !aligned16(Y0) || !aligned16(Y) || !aligned16(ws)) return LOFTQ_ERR_INVALID_ARG;
  const ForwardSpace f = forward_space(ws, n_tok, rows, cols, ad->slots, ad->rank);
  if (ws_bytes < f.bytes) return LOFTQ_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const DropArg d = drop_arg(drop), none = drop_arg(nullptr);
  const PlanView view = plan_view(plan, plan_layout(n_tok, ad->slots));
  const Pool pool = pool_of(ad, d);
  // B in bf16 with whole eights of ranks is read as it lies; else its form is made beside X A^T
  const bool as_it_lies = ad->dt == LOFTQ_BF16 && ad->rank % 8 == 0;
  Prepare prepare{};
  prepare.Bp = as_it_lies ? nullptr : f.Bp;
  prepare.rows = rows;
  prepare.cols = cols;
  // Many tokens: the partials are added once, beside the making of B's form, and not by every workgroup that reads
  // them (2048 tokens, rank 64 in fp32: 84 us without); few tokens save the launch.
  const bool added = n_tok > kFewAdapterTokens;
  AdapterDownJobs down{};
  down.job[1] = AdapterDown{static_cast<const __bf16*>(X), cols, ad->A, ad->rank * cols, false, f.partials, f.ks, 0, d};
  LQ_TRY(launch_adapters_down(down, ad->dt, added ? Prepare{} : prepare, view, pool, s));
  if (added) LQ_TRY(launch_adapters_sum(AdapterSumJobs{{{f.partials, f.ks, f.H, nullptr}, {}}}, prepare, view, pool, s));
  AdapterUp up{added ? f.H : f.partials, added ? 1 : f.ks, rows, as_it_lies ? static_cast<const __bf16*>(ad->B) : f.Bp,
               as_it_lies ? ad->rank : pool.rp, !as_it_lies, Y0, Y, ydt, none};
  return from_hip(launch_adapters_up(up, view, pool, s));
}

size_t loftq_adapters_backward_workspace_bytes(int64_t n_tok, int64_t rows, int64_t cols, int32_t slots, int32_t rank) {
  return query_ok(n_tok, rows, cols, slots, rank, true) && n_tok > 0 ? backward_space(nullptr, n_tok, rows, cols, slots, rank).bytes
                                                                     : 0;
}

loftq_status_t loftq_adapters_backward(const void* dY, const void* X, int64_t n_tok, int64_t rows, int64_t cols,
                                       const loftq_adapters_t* ad, const int32_t* plan, size_t plan_bytes,
                                       const loftq_dropout_t* drop, const void* dX0, void* dX, loftq_dtype_t xdt, float* dB,
                                       float* dA, void* ws, size_t ws_bytes, void* stream) {
  loftq_status_t st = check_call(n_tok, rows, cols, ad, drop);
  if (st != LOFTQ_OK) return st;
  if (dX && !dtype_ok(xdt)) return LOFTQ_ERR_INVALID_ARG;
  if ((dB == nullptr) != (dA == nullptr)) return LOFTQ_ERR_INVALID_ARG;
  if (!dX && !dB && n_tok > 0) return LOFTQ_ERR_INVALID_ARG;   // without tokens dX has no elements and may have no address
  if (!sizes_ok(n_tok, rows, cols, ad->slots, ad->rank, true)) return LOFTQ_ERR_UNSUPPORTED;
  st = check_pool(ad, plan, plan_bytes, n_tok);
  if (st != LOFTQ_OK) return st;
  if (!aligned16(dX0) || !aligned16(dX) || !aligned16(dB) || !aligned16(dA)) return LOFTQ_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const DropArg d = drop_arg(drop), none = drop_arg(nullptr);
  const PlanView view = plan_view(plan, plan_layout(n_tok, ad->slots));
  const Pool pool = pool_of(ad, d);
  if (n_tok == 0) {   // sums over no tokens
    if (dB) LQ_TRY(launch_adapters_grad_sum(AdapterGradJobs{{{nullptr, nullptr, nullptr, dB, rows, rows, none}, {nullptr, nullptr, nullptr, dA, cols, cols, none}}}, view, pool, s));
    return LOFTQ_OK;
  }
  if (!dY || !ws || !aligned16(dY) || !aligned16(ws)) return LOFTQ_ERR_INVALID_ARG;
  if (dB && (!X || !aligned16(X))) return LOFTQ_ERR_INVALID_ARG;
  const BackwardSpace f = backward_space(ws, n_tok, rows, cols, ad->slots, ad->rank);
  if (ws_bytes < f.bytes) return LOFTQ_ERR_WORKSPACE;
  const i64 rows8 = pad8(rows);
  const __bf16* G = static_cast<const __bf16*>(dY);
  const __bf16* Xb = static_cast<const __bf16*>(X);
  if (f.G != nullptr) {
    LQ_TRY(launch_adapters_pad(G, f.G, n_tok, rows, rows8, s));
    G = f.G;
  }
  const bool a_as_it_lies = ad->dt == LOFTQ_BF16;
  Prepare prepare{};
  prepare.Bt = f.Bt;
  prepare.Ab = dB && !a_as_it_lies ? f.Ab : nullptr;
  prepare.dB = dB;
  prepare.dA = dA;
  prepare.rows = rows;
  prepare.rows8 = rows8;
  prepare.cols = cols;
  LQ_TRY(launch_adapters_prepare(prepare, view, pool, s));
  Prepare later{};   // A's columns are wanted last: their form is made beside the sums
  later.At = dX ? f.At : nullptr;
  later.rows = rows;
  later.rows8 = rows8;
  later.cols = cols;
  // P = G B for dX and dA, H = keep(X) A^T for dB
  AdapterDownJobs down{{{G, rows8, f.Bt, pool.rp * rows8, true, f.down_p, f.ks_p, 0, none}, {}}};
  AdapterSumJobs sum{{{f.down_p, f.ks_p, dX ? f.P : nullptr, dB ? f.Pt : nullptr}, {}}};
  if (dB) {
    down.job[1] = a_as_it_lies ? AdapterDown{Xb, cols, ad->A, ad->rank * cols, false, f.down_h, f.ks_h, 0, d}
                               : AdapterDown{Xb, cols, f.Ab, pool.rp * cols, true, f.down_h, f.ks_h, 0, d};
    sum.job[1] = AdapterSum{f.down_h, f.ks_h, nullptr, f.Ht};
  }
  LQ_TRY(launch_adapters_down(down, LOFTQ_BF16, Prepare{}, view, pool, s));
  LQ_TRY(launch_adapters_sum(sum, later, view, pool, s));
  if (dB) {
    const AdapterGradJobs grad{{{G, f.Ht, f.grad_b, dB, rows8, rows, none}, {Xb, f.Pt, f.grad_a, dA, cols, cols, d}}};
    LQ_TRY(launch_adapters_grad(grad, view, pool, s));
    if (plan_layout(n_tok, ad->slots).max_parts > 0) LQ_TRY(launch_adapters_grad_sum(grad, view, pool, s));
  }
  if (!dX) return LOFTQ_OK;
  return from_hip(launch_adapters_up(AdapterUp{f.P, 1, cols, f.At, pool.rp, true, dX0, dX, xdt, d}, view, pool, s));
}

}  // extern "C"
