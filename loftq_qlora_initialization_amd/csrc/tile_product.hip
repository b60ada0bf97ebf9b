// The tiled product of the adapted layer on the matrix cores: C = X W^T + gain keep S V^T
// for operands whose K runs along their rows, in bf16 or in MXFP4.
//
// A K step is 128 bytes of a row in either format (64 bf16 or 256 FP4 values) and a lane's
// operand of one matrix instruction 16 bytes, so both formats share every address: for
// v_mfma_f32_32x32x16_bf16 lane L supplies row L%32, k = 8 (L/32) .. + 7, for
// v_mfma_scale_f32_32x32x64_f8f6f4 row L%32, k = 32 (L/32) .. + 31, one whole MXFP4 block,
// whose scale byte the instruction applies.  The weight is the first operand, so lane L
// receives token L%32, features 8 (v/4) + 4 (L/32) + v%4 in element v: four consecutive
// features a quad.
//
// A workgroup owns TM tokens x TN features.  Each step's rows go straight from memory to
// LDS (16 bytes a lane), double buffered with one barrier a step: the next step's loads
// are in flight while this one is multiplied.  16-byte piece c of LDS row i lies at place
// c ^ (i & 7), so that the 32 rows an operand load reads at one k spread over all banks.
#include "layer.h"

#include <type_traits>

namespace loftq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 128;

template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (N > 0) {
    static_for<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

__device__ __forceinline__ i32x8 widen(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// Workgroups are dealt to the 8 XCDs round-robin by id; each XCD gets a contiguous run of
// tiles.  Within a run, kBand token tiles by all features in turn, tokens inner, so that
// the rows a band shares stay in the XCD's L2.
constexpr int64_t kBand = 8;
__device__ __forceinline__ void tile_of(int64_t wg, int64_t ntm, int64_t ntn, int64_t& tm, int64_t& tn) {
  const int64_t total = ntm * ntn, per = total / 8;
  const int64_t t = wg < per * 8 ? (wg % 8) * per + wg / 8 : wg;
  const int64_t band = t / (kBand * ntn), first = band * kBand;
  const int64_t height = ntm - first < kBand ? ntm - first : kBand;
  const int64_t in = t - band * kBand * ntn;
  tm = first + in % height;
  tn = in / height;
}

template <bool kMx, int TM, int TN, int WM, int WN, typename O>
__global__ __launch_bounds__((TM / WM) * (TN / WN) * 64) void tile_product_kernel(TileProduct t) {
  constexpr int kThreads = (TM / WM) * (TN / WN) * 64;
  constexpr int kWavesM = TM / WM;
  constexpr int MT = WM / 32, NT = WN / 32;   // 32 x 32 tiles of a wave
  constexpr int kRows = TM + TN;              // LDS rows: features, then tokens
  constexpr int kLoads = kRows * 8 / kThreads;
  static_assert(kRows * 8 % kThreads == 0, "whole 16-byte pieces per thread");
  __shared__ __align__(16) char lds[2 * kRows * kStepBytes];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w % kWavesM, wn = w / kWavesM;
  const int li = lane & 31, lh = lane >> 5;
  const int64_t ntm = (t.M + TM - 1) / TM, ntn = (t.N + TN - 1) / TN;
  int64_t tm, tn;
  tile_of(blockIdx.x, ntm, ntn, tm, tn);
  const int64_t m0 = tm * TM, n0 = tn * TN;

  // this thread's pieces of a step; rows past the last repeat it (loaded, never stored)
  const char* src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = i * kThreads + tid, row = c >> 3, piece = (c & 7) ^ (row & 7);
    if (row < TN) {
      const int64_t n = n0 + row < t.N ? n0 + row : t.N - 1;
      src[i] = static_cast<const char*>(t.W) + n * t.ldw + piece * 16;
    } else {
      const int64_t m = m0 + row - TN < t.M ? m0 + row - TN : t.M - 1;
      src[i] = static_cast<const char*>(t.X) + m * t.ldx + piece * 16;
    }
  }
  auto stage = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)src[i],
          (__attribute__((address_space(3))) void*)(lds + buf * kRows * kStepBytes + (i * kThreads + w * 64) * 16), 16, 0, 0);
      src[i] += kStepBytes;
    }
  };

  f32x16 acc[NT][MT];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;

  // MXFP4: each lane's 8 scale bytes of its rows for the step being multiplied; the
  // operand of matrix instruction kk covers blocks 2 kk + L/32, so byte kk of `sel`
  const u32x2* wsc[kMx ? NT : 1];
  const u32x2* xsc[kMx ? MT : 1];
  u32x2 wnext[kMx ? NT : 1], xnext[kMx ? MT : 1];
  const uint32_t sel = lh ? 0x07050301u : 0x06040200u;
  if constexpr (kMx) {
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int64_t n = n0 + wn * WN + a * 32 + li;
      wsc[a] = reinterpret_cast<const u32x2*>(t.wscale) + (n < t.N ? n : t.N - 1);
      wnext[a] = *wsc[a];
    }
#pragma unroll
    for (int b = 0; b < MT; ++b) {
      const int64_t m = m0 + wm * WM + b * 32 + li;
      xsc[b] = reinterpret_cast<const u32x2*>(t.xscale) + (m < t.M ? m : t.M - 1);
      xnext[b] = *xsc[b];
    }
  }

  stage(0);
  for (int k = 0; k < t.steps; ++k) {
    const char* tile = lds + (k & 1) * kRows * kStepBytes;
    __syncthreads();   // step k has landed, and every wave has left the other buffer
    uint32_t ws[kMx ? NT : 1], xs[kMx ? MT : 1];
    if constexpr (kMx) {
#pragma unroll
      for (int a = 0; a < NT; ++a) ws[a] = __builtin_amdgcn_perm(wnext[a][1], wnext[a][0], sel);
#pragma unroll
      for (int b = 0; b < MT; ++b) xs[b] = __builtin_amdgcn_perm(xnext[b][1], xnext[b][0], sel);
    }
    if (k + 1 < t.steps) {
      stage((k + 1) & 1);
      if constexpr (kMx) {
#pragma unroll
        for (int a = 0; a < NT; ++a) wnext[a] = *(wsc[a] += t.N);
#pragma unroll
        for (int b = 0; b < MT; ++b) xnext[b] = *(xsc[b] += t.M);
      }
    }
    static_for<4>([&](auto kk_) __attribute__((always_inline)) {
      constexpr int kk = decltype(kk_)::value;
      i32x4 wf[NT], xf[MT];
#pragma unroll
      for (int a = 0; a < NT; ++a) {
        const int row = wn * WN + a * 32 + li;
        wf[a] = *reinterpret_cast<const i32x4*>(tile + row * kStepBytes + (((2 * kk + lh) ^ (row & 7)) << 4));
      }
#pragma unroll
      for (int b = 0; b < MT; ++b) {
        const int row = TN + wm * WM + b * 32 + li;
        xf[b] = *reinterpret_cast<const i32x4*>(tile + row * kStepBytes + (((2 * kk + lh) ^ (row & 7)) << 4));
      }
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b) {
          if constexpr (kMx)
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(wf[a]), widen(xf[b]), acc[a][b], 4, 4, kk,
                                                                         static_cast<int>(ws[a]), kk,
                                                                         static_cast<int>(xs[b]));
          else
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wf[a]),
                                                                __builtin_bit_cast(bf16x8, xf[b]), acc[a][b], 0, 0, 0);
        }
    });
  }

  const uint64_t key = t.drop.thr != 0 ? drop_key(t.drop) : 0;
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b) {
      const int64_t m = m0 + wm * WM + b * 32 + li, nb = n0 + wn * WN + a * 32;
      f32x16 lora;
#pragma unroll
      for (int v = 0; v < 16; ++v) lora[v] = 0.f;
      if (t.V != nullptr) {
        const int64_t vr = nb + li < t.N ? nb + li : t.N - 1, sr = m < t.M ? m : t.M - 1;
        for (int p = 0; p < t.rp; p += 16) {
          const bf16x8 v = *reinterpret_cast<const bf16x8*>(t.V + vr * t.rp + p + 8 * lh);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            lora = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                v, *reinterpret_cast<const bf16x8*>(t.S + (sr * 3 + q) * t.rp + p + 8 * lh), lora, 0, 0, 0);
        }
      }
      if (m >= t.M) continue;
      O* out = static_cast<O*>(t.out) + m * t.N;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = nb + 8 * q + 4 * lh;
        float y[4];
        // the mask's word of four features; it is only asked for where N % 4 == 0
        const uint64_t word = t.drop.thr != 0 ? drop_word(key, static_cast<uint64_t>(m * t.N + n) >> 2) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float l = t.drop.thr == 0 || drop_keeps(word, j, t.drop.thr) ? lora[4 * q + j] : 0.f;
          y[j] = t.V != nullptr ? fmaf(t.gain, l, acc[a][b][4 * q + j]) : acc[a][b][4 * q + j];
        }
        if (t.N % 4 == 0) {
          if (n < t.N) {
            if constexpr (sizeof(O) == 4)
              *reinterpret_cast<f32x4*>(out + n) = f32x4{y[0], y[1], y[2], y[3]};
            else
              *reinterpret_cast<bf16x4*>(out + n) =
                  bf16x4{static_cast<__bf16>(y[0]), static_cast<__bf16>(y[1]), static_cast<__bf16>(y[2]),
                         static_cast<__bf16>(y[3])};
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < t.N) out[n + j] = static_cast<O>(y[j]);
        }
      }
    }
}

template <bool kMx, int TM, int TN, int WM, int WN>
hipError_t launch_tile(const TileProduct& t, hipStream_t s) {
  const int64_t wgs = ((t.M + TM - 1) / TM) * ((t.N + TN - 1) / TN);
  const dim3 grid(static_cast<unsigned>(wgs)), block((TM / WM) * (TN / WN) * 64);
  if (t.odt == LOFTQ_BF16)
    LQ_LAUNCH(kMx ? "mx_product" : "bf16_product", (tile_product_kernel<kMx, TM, TN, WM, WN, __bf16>), grid, block, 0, s, t);
  else
    LQ_LAUNCH(kMx ? "mx_product" : "bf16_product", (tile_product_kernel<kMx, TM, TN, WM, WN, float>), grid, block, 0, s, t);
  return hipGetLastError();
}

}  // namespace

bool tile_product_shape_ok(int64_t M, int64_t N) {
  // one launch has at most 2^32 work-items: 256 per 128 x 128 outputs
  return ((M + 127) / 128) * ((N + 127) / 128) < (int64_t(1) << 24);
}

hipError_t launch_tile_product(const TileProduct& t, bool mx, hipStream_t s) {
  return mx ? launch_tile<true, 128, 128, 64, 64>(t, s) : launch_tile<false, 128, 128, 64, 64>(t, s);
}

}  // namespace loftq
