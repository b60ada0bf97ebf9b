// Dropout Y = X mask / (1 - p) over a flat array, and its gradient (the same map of
// the gradient, with the same mask).
//
// Bound by memory: 16 bytes in and out a thread, whose mask's words (two for bf16, one for
// fp32) hide behind them.  8192 x 11008 bf16: 63.9 us, 5.65 TB/s (an elementwise product of
// 4 GiB reaches 6.27); one token of 4096: 2 us of kernel, the rest of its 6 us the call from Python.
#include "dropout.h"
#include "internal.h"

namespace loftq {
namespace {

constexpr int kDropThreads = 256;

template <typename T>
__device__ __forceinline__ T drop_one(T x, bool keep, float scale) {
  return keep ? static_cast<T>(static_cast<float>(x) * scale) : static_cast<T>(0.f);
}

// One thread per 16 bytes (8 bf16 or 4 fp32 elements); the first thread takes the
// elements past the last whole 16 bytes one by one.  Y may be X: each element is read and
// written by one thread, in that order.
template <typename T>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const T* X, int64_t n, DropArg d, T* Y) {
  constexpr int E = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(E)));
  const uint64_t key = drop_key(d);
  const int64_t nv = n / E;
  for (int64_t v = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x; v < nv;
       v += static_cast<int64_t>(gridDim.x) * kDropThreads) {
    const vec x = reinterpret_cast<const vec*>(X)[v];
    vec y;
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      const uint64_t word = drop_word(key, static_cast<uint64_t>(v) * (E / 4) + q);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[4 * q + j] = drop_one<T>(x[4 * q + j], drop_keeps(word, j, d.thr), d.scale);
    }
    reinterpret_cast<vec*>(Y)[v] = y;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    for (int64_t i = nv * E; i < n; ++i)
      Y[i] = drop_one<T>(X[i], drop_keeps(drop_word(key, static_cast<uint64_t>(i) >> 2), static_cast<int>(i & 3), d.thr),
                         d.scale);
  }
}

}  // namespace

hipError_t launch_dropout(const void* X, loftq_dtype_t dt, int64_t n, const DropArg& d, void* Y, hipStream_t s) {
  const int64_t per = dt == LOFTQ_BF16 ? 8 : 4;
  int64_t wgs = (n / per + kDropThreads - 1) / kDropThreads;
  wgs = wgs < 1 ? 1 : (wgs > 8192 ? 8192 : wgs);
  const dim3 grid(static_cast<unsigned>(wgs));
  if (dt == LOFTQ_BF16)
    LQ_LAUNCH("dropout", (dropout_kernel<__bf16>), grid, dim3(kDropThreads), 0, s, static_cast<const __bf16*>(X), n, d,
              static_cast<__bf16*>(Y));
  else
    LQ_LAUNCH("dropout", (dropout_kernel<float>), grid, dim3(kDropThreads), 0, s, static_cast<const float*>(X), n, d,
              static_cast<float*>(Y));
  return hipGetLastError();
}

}  // namespace loftq
