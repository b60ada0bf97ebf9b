// MXFP4 quantization (optionally of a residual W - B A) and dequantization.
//
// Without an adapter both are bound by memory: 11008 x 4096 fp32 to codes 42 us (204 MB, 4.9
// TB/s), codes and W to the fp32 residual 61 us (385 MB, 6.3 TB/s).  Neighbouring threads take
// neighbouring 16 or 32 bytes of a row; the codes of a thread are one word, so no LDS is needed.
// A residual's r products run on the vector units and the rows of A come from the caches; they,
// not memory, set its time (11008 x 4096 bf16, traced: 60 us at r = 16, 160 us at r = 64).
#include "internal.h"
#include "mxfp4.h"

namespace loftq {
namespace {

constexpr int kMxThreads = 256;

// Eight elements of a row whose address is a multiple of their size only: rows of any length
// are read and written in whole vectors (the memory system takes them at any address).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  T v[8];
  __builtin_memcpy(v, p, sizeof v);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(v[j]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  T v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = static_cast<T>(x[j]);
  __builtin_memcpy(p, v, sizeof v);
}

// One thread per 8 consecutive columns of kRows rows of the padded matrix: one row of W, or
// four of a residual R = W - B A, which share each load of A: calls over 11008 x 4096 bf16 with
// 1, 2, 4 and 8 rows took 117, 71, 58 and 66 us at r = 16, and 419, 258, 175 and 172 us at r = 64 (8192 x
// 28672: 2227, 1321, 864 and 963 us).  R is formed in fp32, the r products added in the order of p.
template <typename T, int kRows>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(const T* __restrict__ W, int64_t rows, int64_t cols,
                                                                 int64_t steps, const float* __restrict__ B,
                                                                 const float* __restrict__ A, int r,
                                                                 uint8_t* __restrict__ packed,
                                                                 uint8_t* __restrict__ scales) {
  const uint32_t id = blockIdx.x * kMxThreads + threadIdx.x;   // below 2^32
  const uint32_t per_row = static_cast<uint32_t>(steps * (kMxStep / 8));
  const int64_t row0 = static_cast<int64_t>(id / per_row) * kRows, c0 = static_cast<int64_t>(id % per_row) * 8;
  if (row0 >= rows) return;   // whole quads: per_row % 32 == 0
  const bool whole = c0 + 8 <= cols;
  float x[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {   // rows past the last repeat it and are not stored
    const T* src = W + (row0 + i < rows ? row0 + i : rows - 1) * cols + c0;
    if (whole) {
      load8(src, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = c0 + j < cols ? static_cast<float>(src[j]) : 0.f;
    }
  }
  if constexpr (kRows > 1) {
    float ba[kRows][8] = {};
    for (int p = 0; p < r; ++p) {
      float a[8];
      const float* src = A + static_cast<int64_t>(p) * cols + c0;
      if (whole) {
        load8(src, a);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = c0 + j < cols ? src[j] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float b = B[(row0 + i < rows ? row0 + i : rows - 1) * r + p];
#pragma unroll
        for (int j = 0; j < 8; ++j) ba[i][j] = fmaf(b, a[j], ba[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)   // the padding stays zero, also where B is not finite
        if (whole || c0 + j < cols) x[i][j] -= ba[i][j];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t byte;
    const uint32_t word = mx_encode8(x[i], byte);
    const int64_t row = row0 + i;
    if (row >= rows) break;
    *reinterpret_cast<uint32_t*>(packed + row * steps * (kMxStep / 2) + c0 / 2) = word;
    if ((threadIdx.x & 3) == 0) scales[(c0 / kMxStep * rows + row) * 8 + (c0 % kMxStep) / kMxBlock] = static_cast<uint8_t>(byte);
  }
}

// out = deq or W - deq, in fp32 or bf16; one thread per 8 columns.  out may be W: each element is
// read and written by one thread, in that order.
template <typename T, typename O, bool kHasW>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ packed,
                                                                   const uint8_t* __restrict__ scales, int64_t rows,
                                                                   int64_t cols, int64_t steps,
                                                                   const T* W, O* out) {
  const uint32_t id = blockIdx.x * kMxThreads + threadIdx.x;   // below 2^32
  const uint32_t per_row = static_cast<uint32_t>((cols + 7) / 8);
  const int64_t row = id / per_row, c0 = static_cast<int64_t>(id % per_row) * 8;
  if (row >= rows) return;
  const uint32_t word = *reinterpret_cast<const uint32_t*>(packed + row * steps * (kMxStep / 2) + c0 / 2);
  const float sc = mx_scale(scales[(c0 / kMxStep * rows + row) * 8 + (c0 % kMxStep) / kMxBlock]);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fp4_value(word >> (8 * (j >> 1) + (j & 1 ? 0 : 4)) & 15u) * sc;
  const int64_t at = row * cols + c0;
  if (c0 + 8 <= cols) {
    if (kHasW) {
      float w[8];
      load8(W + at, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = w[j] - v[j];
    }
    store8(out + at, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (c0 + j >= cols) break;
    out[at + j] = static_cast<O>(kHasW ? static_cast<float>(W[at + j]) - v[j] : v[j]);
  }
}

unsigned blocks_for(int64_t threads) { return static_cast<unsigned>((threads + kMxThreads - 1) / kMxThreads); }

}  // namespace

bool mx_shape_ok(int64_t rows, int64_t cols) {
  // one launch has a thread per 8 padded columns: at most 2^32 of them
  return rows == 0 || mx_steps(cols) * (kMxStep / 8) <= ((int64_t(1) << 32) - kMxThreads) / rows;
}

hipError_t launch_mx_quantize(const void* W, loftq_dtype_t wdt, int64_t rows, int64_t cols, const float* B,
                              const float* A, int r, uint8_t* packed, uint8_t* scales, hipStream_t s) {
  const int64_t steps = mx_steps(cols);
  const int64_t groups = B != nullptr ? (rows + 3) / 4 : rows;
  const dim3 grid(blocks_for(groups * steps * (kMxStep / 8)));
#define LQ_MXQ(T, ROWS)                                                                                        \
  LQ_LAUNCH("mx_quantize", (mx_quantize_kernel<T, ROWS>), grid, dim3(kMxThreads), 0, s, static_cast<const T*>(W), \
            rows, cols, steps, B, A, r, packed, scales)
  if (wdt == LOFTQ_BF16) {
    if (B != nullptr) LQ_MXQ(__bf16, 4);
    else LQ_MXQ(__bf16, 1);
  } else {
    if (B != nullptr) LQ_MXQ(float, 4);
    else LQ_MXQ(float, 1);
  }
#undef LQ_MXQ
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t cols,
                                const void* W, loftq_dtype_t wdt, void* out, loftq_dtype_t odt, hipStream_t s) {
  const int64_t steps = mx_steps(cols);
  const dim3 grid(blocks_for(rows * ((cols + 7) / 8)));
#define LQ_MXD(T, O, HASW)                                                                                              \
  LQ_LAUNCH("mx_dequantize", (mx_dequantize_kernel<T, O, HASW>), grid, dim3(kMxThreads), 0, s, packed, scales, rows, cols, \
            steps, static_cast<const T*>(W), static_cast<O*>(out))
#define LQ_MXD_O(O)                                            \
  do {                                                         \
    if (W == nullptr) LQ_MXD(float, O, false);                 \
    else if (wdt == LOFTQ_BF16) LQ_MXD(__bf16, O, true);       \
    else LQ_MXD(float, O, true);                               \
  } while (0)
  if (odt == LOFTQ_BF16) LQ_MXD_O(__bf16);
  else LQ_MXD_O(float);
#undef LQ_MXD_O
#undef LQ_MXD
  return hipGetLastError();
}

}  // namespace loftq
