// What the entry points of the adapted layer, of a pool of adapters and of the optimizer share: checks of arguments and the
// division of a workspace.  Host code.
#pragma once

#include <cmath>

#include "dropout.h"
#include "internal.h"

namespace loftq {

bool aligned16(const void* p);
bool shape_ok(int64_t rows, int64_t cols);
loftq_status_t from_hip(hipError_t e);

namespace {

typedef int64_t i64;

// Consecutive 256-byte aligned pieces of a workspace; with a null base it only counts.
struct Arena {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(i64 count) {
    T* p = base != nullptr ? reinterpret_cast<T*>(base + used) : nullptr;
    used += (static_cast<size_t>(count) * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

int rank_pad(int r) { return (r + 15) / 16 * 16; }

bool dtype_ok(loftq_dtype_t t) { return t == LOFTQ_F32 || t == LOFTQ_BF16; }

bool drop_ok(const loftq_dropout_t* d) {
  return d == nullptr || (std::isfinite(d->p) && d->p >= 0.f && d->p <= 1.f &&
                          (reinterpret_cast<uintptr_t>(d->step) & 7u) == 0);
}

DropArg drop_arg(const loftq_dropout_t* d) {
  if (d == nullptr) return DropArg{0, 0, nullptr, 0, 1.f};
  const uint32_t thr = static_cast<uint32_t>(static_cast<double>(d->p) * 65536.0 + 0.5);
  const float scale = thr >= 65536u ? 0.f : static_cast<float>(65536.0 / (65536.0 - thr));
  return DropArg{d->seed, d->offset, d->step, thr, scale};
}

}  // namespace
}  // namespace loftq

#define LQ_TRY(call)                                  \
  do {                                                \
    const hipError_t lq_e_ = (call);                  \
    if (lq_e_ != hipSuccess) return LOFTQ_ERR_HIP;    \
  } while (0)
