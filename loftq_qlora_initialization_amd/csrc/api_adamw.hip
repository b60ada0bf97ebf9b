// C-ABI entry points of the optimizer's step: argument validation, the table's layout, then launches.
#include <algorithm>
#include <cmath>
#include <new>

#include "adamw.h"
#include "entry.h"

using namespace loftq;

namespace {

constexpr int32_t kMostTensors = 65536;
constexpr int64_t kMostElements = int64_t(1) << 36;

// Chunks of all tensors; -1 where there are more elements than a step takes, -2 for a negative length.
int64_t count_chunks(const loftq_adamw_tensor_t* tensors, int32_t count) {
  int64_t chunks = 0, elements = 0;
  for (int32_t i = 0; i < count; ++i) {
    const int64_t n = tensors[i].n;
    if (n < 0) return -2;
    if (n >= kMostElements || (elements += n) >= kMostElements) return -1;
    chunks += adam_chunks(n);
  }
  return chunks < (int64_t(1) << 24) ? chunks : -1;   // a launch has less than 2^32 work-items
}

// Memory that a step reads or writes.
struct Piece {
  uintptr_t begin, end;
  bool written;
};
enum Overlap { kNone, kSome, kUnknown };

// Whether anything that a step writes lies over anything else of it.  Gradients are only read, and may share theirs.
Overlap overlap(const loftq_adamw_tensor_t* tensors, int32_t count, loftq_dtype_t pdt, loftq_dtype_t gdt, int32_t bits,
                const void* table, size_t table_bytes) {
  Piece* const pieces = new (std::nothrow) Piece[static_cast<size_t>(count) * 7 + 1];
  if (pieces == nullptr) return kUnknown;
  Piece* last = pieces;
  auto add = [&](const void* p, int64_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p != nullptr && bytes > 0) *last++ = Piece{at, at + static_cast<uintptr_t>(bytes), written};
  };
  auto size = [](loftq_dtype_t t) { return t == LOFTQ_BF16 ? 2 : 4; };
  for (int32_t i = 0; i < count; ++i) {
    const loftq_adamw_tensor_t& x = tensors[i];
    const int64_t blocks = (x.n + kStateBlock - 1) / kStateBlock;
    add(x.param, x.n * size(pdt), true);
    add(x.grad, x.n * size(gdt), false);
    add(x.m, x.n * (bits / 8), true);
    add(x.v, x.n * (bits / 8), true);
    add(x.copy, x.n * 2, true);
    if (bits == 8) {
      add(x.m_scale, blocks * 4, true);
      add(x.v_scale, blocks * 4, true);
    }
  }
  add(table, static_cast<int64_t>(table_bytes), true);
  std::sort(pieces, last, [](const Piece& a, const Piece& b) { return a.begin < b.begin; });
  uintptr_t written = 0, any = 0;   // where what begins before a piece ends
  Overlap found = kNone;
  for (const Piece* p = pieces; p != last && found == kNone; ++p) {
    if (p->begin < (p->written ? any : written)) found = kSome;
    any = std::max(any, p->end);
    if (p->written) written = std::max(written, p->end);
  }
  delete[] pieces;
  return found;
}

}  // namespace

extern "C" {

size_t loftq_adamw_plan_bytes(const loftq_adamw_tensor_t* tensors, int32_t count) {
  if (count < 0 || count > kMostTensors || (count > 0 && !tensors)) return 0;
  const int64_t chunks = count_chunks(tensors, count);
  return chunks < 0 ? 0 : adam_table(nullptr, count, chunks).bytes;
}

loftq_status_t loftq_adamw_plan(const loftq_adamw_tensor_t* tensors, int32_t count, loftq_dtype_t pdt, loftq_dtype_t gdt,
                                int32_t bits, void* table, size_t table_bytes, loftq_adamw_plan_t* plan, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !dtype_ok(pdt) || !dtype_ok(gdt) || !plan) return LOFTQ_ERR_INVALID_ARG;
  if ((bits != 32 && bits != 8) || count > kMostTensors) return LOFTQ_ERR_UNSUPPORTED;
  const int64_t chunks = count_chunks(tensors, count);
  if (chunks < 0) return chunks == -2 ? LOFTQ_ERR_INVALID_ARG : LOFTQ_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i) {
    const loftq_adamw_tensor_t& x = tensors[i];
    if (!std::isfinite(x.lr_scale) || !std::isfinite(x.weight_decay)) return LOFTQ_ERR_INVALID_ARG;
    if (x.n == 0) continue;
    if (!x.param || !x.grad || !x.m || !x.v) return LOFTQ_ERR_INVALID_ARG;
    if (!aligned16(x.param) || !aligned16(x.grad) || !aligned16(x.m) || !aligned16(x.v) || !aligned16(x.copy)) return LOFTQ_ERR_INVALID_ARG;
    if (bits == 8 && (!x.m_scale || !x.v_scale)) return LOFTQ_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(x.m_scale) & 3u) != 0 || (reinterpret_cast<uintptr_t>(x.v_scale) & 3u) != 0) return LOFTQ_ERR_INVALID_ARG;
  }
  if (!table || !aligned16(table)) return LOFTQ_ERR_INVALID_ARG;
  const AdamTable t = adam_table(table, count, chunks);
  if (table_bytes < t.bytes) return LOFTQ_ERR_WORKSPACE;
  const Overlap o = overlap(tensors, count, pdt, gdt, bits, table, t.bytes);   // steps would race
  if (o != kNone) return o == kSome ? LOFTQ_ERR_INVALID_ARG : LOFTQ_ERR_HIP;
  *plan = loftq_adamw_plan_t{table, chunks, count, bits, pdt, gdt};
  return from_hip(launch_adamw_table(tensors, count, t, static_cast<hipStream_t>(stream)));
}

loftq_status_t loftq_adamw(const loftq_adamw_plan_t* plan, const loftq_adamw_t* step, float* norm, void* stream) {
  if (!plan || !step || !plan->table || plan->chunks < 0 || plan->count < 0) return LOFTQ_ERR_INVALID_ARG;
  auto share = [](double b) { return b >= 0.0 && b < 1.0; };
  if (!std::isfinite(step->lr) || step->lr < 0.0 || !share(step->beta1) || !share(step->beta2)) return LOFTQ_ERR_INVALID_ARG;
  if (!std::isfinite(step->eps) || !(static_cast<float>(step->eps) > 0.f)) return LOFTQ_ERR_INVALID_ARG;
  if (!std::isfinite(step->max_norm) || step->max_norm < 0.0 || step->t < 1) return LOFTQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(step->step) & 7u) != 0 || (reinterpret_cast<uintptr_t>(step->lr_factor) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(norm) & 3u) != 0)
    return LOFTQ_ERR_INVALID_ARG;
  if (norm != nullptr && step->max_norm == 0.0) return LOFTQ_ERR_INVALID_ARG;   // no norm is formed
  if (plan->chunks == 0 && norm == nullptr) return LOFTQ_OK;
  const AdamTable t = adam_table(const_cast<void*>(plan->table), plan->count, plan->chunks);
  return from_hip(launch_adamw(*plan, t, *step, norm, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
