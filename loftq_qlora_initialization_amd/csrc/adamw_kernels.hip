// AdamW over many tensors in one launch, with states in fp32 or in 8 bits.
//
// A workgroup takes a chunk of one tensor, a wave four blocks of 256 elements of it, four
// elements a lane: a block of 8-bit states is one wave's, so its largest magnitude is found
// by exchanges within the wave and its scale is read and written once.
//
// Bound by memory: every number is read once and written once, gradients that are clipped are read twice (the
// norm has to be known first).  Of 40 million elements the step with fp32 states moves 1.12 GB in 192 us (5.8 TB/s)
// and the norm 0.16 GB in about 50; of 160 million with 8-bit states, fp32 parameters and a bf16 copy the step
// moves 2.9 GB in 540 to 555 us (5.3 TB/s) and the norm 0.64 GB in 150.  Elements of one tensor in a chunk keep a workgroup's
// scalars the same; 4096 of them are four loads a lane and give one layer's factors 305 workgroups.
#include <cmath>

#include "adamw.h"
#include "reduce.h"

namespace loftq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64, kPerTable = 32;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct TableArgs {
  loftq_adamw_tensor_t tensor[kPerTable];
  int64_t chunk[kPerTable];   // a tensor's first
  int32_t first;
};

__global__ __launch_bounds__(kThreads) void table_kernel(TableArgs a, AdamTable t) {
  const int i = blockIdx.x;
  const loftq_adamw_tensor_t& x = a.tensor[i];
  if (threadIdx.x == 0) t.tensors[a.first + i] = x;
  const int64_t chunks = (x.n + kChunk - 1) / kChunk;
  for (int64_t c = threadIdx.x; c < chunks; c += kThreads)
    t.chunks[a.chunk[i] + c] = make_int2(a.first + i, static_cast<int>(c));
}

// Four elements of a lane; `left` of them exist.
template <typename T>
__device__ __forceinline__ void load4(const void* from, int64_t at, int left, float (&x)[4]) {
  typedef T vec __attribute__((ext_vector_type(4)));
  const T* p = static_cast<const T*>(from) + at;
  if (left >= 4) {
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = static_cast<float>(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = j < left ? static_cast<float>(p[j]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(void* to, int64_t at, int left, const float (&x)[4]) {
  typedef T vec __attribute__((ext_vector_type(4)));
  T* p = static_cast<T*>(to) + at;
  if (left >= 4) {
    vec v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = static_cast<T>(x[j]);
    *reinterpret_cast<vec*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = static_cast<T>(x[j]);
  }
}
__device__ __forceinline__ uint32_t load_codes(const void* from, int64_t at, int left) {
  const uint8_t* p = static_cast<const uint8_t*>(from) + at;
  if (left >= 4) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) w |= static_cast<uint32_t>(p[j]) << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes(void* to, int64_t at, int left, uint32_t w) {
  uint8_t* p = static_cast<uint8_t*>(to) + at;
  if (left >= 4) {
    *reinterpret_cast<uint32_t*>(p) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) p[j] = static_cast<uint8_t>(w >> (8 * j));
}

// The largest magnitude of a block, as its bits: an infinity or a NaN is larger than any number.
__device__ __forceinline__ uint32_t block_amax(const float (&x)[4]) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7FFFFFFFu;
    a = b > a ? b : a;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(a, d);
    a = o > a ? o : a;
  }
  return a;
}
// A block's scale for values up to `top`, and its inverse (0 where the scale is 0).  The scale is a product with the
// rounded inverse, up to 2^-23 off the quotient: the codes are the nearest for this scale, so either serves (697 us
// against 699 for 32 layers at rank 64 with a division), and this one is the header's definition.
__device__ __forceinline__ float block_scale(uint32_t amax, float top, double& inverse) {
  if (amax >= 0x7F800000u) {
    const float nan = __uint_as_float(0x7FC00000u);
    inverse = nan;
    return nan;
  }
  if (amax < 0x0D800000u) {   // 2^-100
    inverse = 0.0;
    return 0.f;
  }
  const float scale = __uint_as_float(amax) * (1.f / top);
  inverse = 1.0 / static_cast<double>(scale);
  return scale;
}
// x in fp32 with its last bit set where it is not exact, so that rounding to fewer bits afterwards goes by x itself.
__device__ __forceinline__ float to_odd(double x) {
  const float f = static_cast<float>(x);
  const double rest = x - static_cast<double>(f);
  uint32_t b = __float_as_uint(f);
  if (rest != 0.0) b = (fabs(static_cast<double>(f)) > fabs(x) ? b - 1 : b) | 1u;   // a NaN's rest is not 0: it stays one
  return __uint_as_float(b);
}

// sum of the squares of all gradients, a part per workgroup
template <typename G>
__global__ __launch_bounds__(kThreads) void norm_kernel(AdamTable t, int64_t chunks) {
  __shared__ double part[kWaves];
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int2 at = t.chunks[c];
    const loftq_adamw_tensor_t& x = t.tensors[at.x];
    const int64_t begin = static_cast<int64_t>(at.y) * kChunk + threadIdx.x * 4;
    constexpr int kLoads = kChunk / (4 * kThreads);
    float g[kLoads][4];
    if (static_cast<int64_t>(at.y + 1) * kChunk <= x.n) {   // a whole chunk: every load in flight at once
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load4<G>(x.grad, begin + i * (4 * kThreads), 4, g[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int64_t left = x.n - begin - i * (4 * kThreads);
        load4<G>(x.grad, begin + i * (4 * kThreads), left < 0 ? 0 : (left < 4 ? static_cast<int>(left) : 4), g[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = fma(static_cast<double>(g[i][j]), static_cast<double>(g[i][j]), sum);
  }
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kWaves; ++w) s += part[w];
    t.partials[blockIdx.x] = s;
  }
}

// What a step's elements share, formed on the device where it depends on device memory.
__global__ __launch_bounds__(kThreads) void scalars_kernel(AdamTable t, loftq_adamw_t step, int partials, float* norm_out) {
  double norm = 0.0;   // of no elements
  if (partials > 0) norm = sqrt(block_sum_fixed(t.partials, partials));
  if (threadIdx.x != 0) return;
  int64_t at = step.t + (step.step != nullptr ? *step.step : 0);
  if (at < 1) at = 1;
  AdamScalars s{};
  s.lr = step.lr * (step.lr_factor != nullptr ? static_cast<double>(*step.lr_factor) : 1.0);
  s.bias1 = 1.0 - pow(step.beta1, static_cast<double>(at));
  s.root2 = 1.0 / sqrt(1.0 - pow(step.beta2, static_cast<double>(at)));
  s.clip = 1.0;
  if (step.max_norm > 0.0) {
    const double c = step.max_norm / (norm + 1e-6);
    s.clip = !isfinite(norm) ? -1.0 : (c < 1.0 ? c : 1.0);
    if (norm_out != nullptr) *norm_out = static_cast<float>(norm);
  }
  *t.scalars = s;
}

template <typename P, typename G, bool k8Bit>
__global__ __launch_bounds__(kThreads) void step_kernel(AdamTable t, AdamScalars host, bool on_device, AdamDecays d) {
  const AdamScalars s = on_device ? *t.scalars : host;
  if (s.clip < 0.0) return;
  const int2 at = t.chunks[blockIdx.x];
  const loftq_adamw_tensor_t x = t.tensors[at.x];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const double lr = s.lr * static_cast<double>(x.lr_scale);
  const float shrink = static_cast<float>(1.0 - lr * static_cast<double>(x.weight_decay));
  const float size = static_cast<float>(lr / s.bias1), root2 = static_cast<float>(s.root2);
#pragma unroll
  for (int i = 0; i < kChunk / (kWaves * kStateBlock); ++i) {
    const int64_t block = static_cast<int64_t>(at.y) * (kChunk / kStateBlock) + i * kWaves + w;
    const int64_t e = block * kStateBlock + lane * 4, rest = x.n - e;
    if (block * kStateBlock >= x.n) return;   // the whole wave
    const int left = rest < 0 ? 0 : (rest < 4 ? static_cast<int>(rest) : 4);
    float p[4], g[4], m[4], v[4];
    load4<P>(x.param, e, left, p);
    load4<G>(x.grad, e, left, g);
    double m8[4], v8[4];   // with states in 8 bits: what the codes are the nearest to
    if constexpr (k8Bit) {
      const uint32_t mc = load_codes(x.m, e, left), vc = load_codes(x.v, e, left);
      const double ms = x.m_scale[block], vs = x.v_scale[block];
      m8[0] = __builtin_amdgcn_cvt_f32_fp8(mc, 0) * ms;
      m8[1] = __builtin_amdgcn_cvt_f32_fp8(mc, 1) * ms;
      m8[2] = __builtin_amdgcn_cvt_f32_fp8(mc, 2) * ms;
      m8[3] = __builtin_amdgcn_cvt_f32_fp8(mc, 3) * ms;
      v8[0] = __builtin_amdgcn_cvt_f32_bf8(vc, 0) * vs;
      v8[1] = __builtin_amdgcn_cvt_f32_bf8(vc, 1) * vs;
      v8[2] = __builtin_amdgcn_cvt_f32_bf8(vc, 2) * vs;
      v8[3] = __builtin_amdgcn_cvt_f32_bf8(vc, 3) * vs;
    } else {
      load4<float>(x.m, e, left, m);
      load4<float>(x.v, e, left, v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (k8Bit) {   // in fp64: a rounding to fp32 in between would move values over the codes' borders
        const double gj = s.clip * static_cast<double>(g[j]);
        m8[j] = d.b1 * m8[j] + d.c1 * gj;
        v8[j] = d.b2 * v8[j] + (d.c2 * gj) * gj;
        m[j] = static_cast<float>(m8[j]);
        v[j] = static_cast<float>(v8[j]);
      } else {
        const float gj = static_cast<float>(s.clip) * g[j];
        m[j] = static_cast<float>(d.b1) * m[j] + static_cast<float>(d.c1) * gj;
        v[j] = static_cast<float>(d.b2) * v[j] + (static_cast<float>(d.c2) * gj) * gj;
      }
      p[j] = p[j] * shrink - size * (m[j] / (sqrtf(v[j]) * root2 + d.eps));
    }
    store4<P>(x.param, e, left, p);
    if (x.copy != nullptr) store4<__bf16>(x.copy, e, left, p);
    if constexpr (k8Bit) {
      double mi, vi;   // inverse scales
      const float ms = block_scale(block_amax(m), 448.f, mi), vs = block_scale(block_amax(v), 57344.f, vi);
      uint32_t mc = 0, vc = 0;
      mc = __builtin_amdgcn_cvt_pk_fp8_f32(to_odd(m8[0] * mi), to_odd(m8[1] * mi), mc, false);
      mc = __builtin_amdgcn_cvt_pk_fp8_f32(to_odd(m8[2] * mi), to_odd(m8[3] * mi), mc, true);
      vc = __builtin_amdgcn_cvt_pk_bf8_f32(to_odd(v8[0] * vi), to_odd(v8[1] * vi), vc, false);
      vc = __builtin_amdgcn_cvt_pk_bf8_f32(to_odd(v8[2] * vi), to_odd(v8[3] * vi), vc, true);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v8[j] > 0.0 && vi > 0.0 && (vc >> (8 * j) & 255u) == 0) vc |= 1u << (8 * j);   // fl(v8) may be 0
      store_codes(x.m, e, left, mc);
      store_codes(x.v, e, left, vc);
      if (lane == 0) {
        x.m_scale[block] = ms;
        x.v_scale[block] = vs;
      }
    } else {
      store4<float>(x.m, e, left, m);
      store4<float>(x.v, e, left, v);
    }
  }
}

}  // namespace

hipError_t launch_adamw_table(const loftq_adamw_tensor_t* tensors, int32_t count, const AdamTable& t, hipStream_t s) {
  int64_t chunk = 0;
  for (int32_t first = 0; first < count; first += kPerTable) {
    TableArgs a{};
    a.first = first;
    const int here = count - first < kPerTable ? count - first : kPerTable;
    for (int i = 0; i < here; ++i) {
      a.tensor[i] = tensors[first + i];
      a.chunk[i] = chunk;
      chunk += adam_chunks(tensors[first + i].n);
    }
    LQ_LAUNCH("adamw_table", table_kernel, dim3(here), dim3(kThreads), 0, s, a, t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw(const loftq_adamw_plan_t& plan, const AdamTable& t, const loftq_adamw_t& step, float* norm, hipStream_t s) {
  const bool clip = step.max_norm > 0.0, on_device = clip || step.step != nullptr || step.lr_factor != nullptr;
  AdamScalars host{};
  if (on_device) {
    const int parts = !clip ? 0 : static_cast<int>(plan.chunks < kNormWorkgroups ? plan.chunks : kNormWorkgroups);
    if (parts > 0) {
      if (plan.gdt == LOFTQ_BF16) LQ_LAUNCH("adamw_norm", norm_kernel<__bf16>, dim3(parts), dim3(kThreads), 0, s, t, plan.chunks);
      else LQ_LAUNCH("adamw_norm", norm_kernel<float>, dim3(parts), dim3(kThreads), 0, s, t, plan.chunks);
    }
    LQ_LAUNCH("adamw_scalars", scalars_kernel, dim3(1), dim3(kThreads), 0, s, t, step, parts, norm);
  } else {
    host.lr = step.lr;
    host.bias1 = 1.0 - std::pow(step.beta1, static_cast<double>(step.t));
    host.root2 = 1.0 / std::sqrt(1.0 - std::pow(step.beta2, static_cast<double>(step.t)));
    host.clip = 1.0;
  }
  if (plan.chunks == 0) return hipGetLastError();
  const AdamDecays d{step.beta1, 1.0 - step.beta1, step.beta2, 1.0 - step.beta2, static_cast<float>(step.eps)};
  const dim3 grid(static_cast<unsigned>(plan.chunks)), block(kThreads);
#define LQ_STEP(P, G, E) LQ_LAUNCH("adamw_step", (step_kernel<P, G, E>), grid, block, 0, s, t, host, on_device, d)
#define LQ_STEP_G(P, G)               \
  do {                                \
    if (plan.bits == 8) LQ_STEP(P, G, true); \
    else LQ_STEP(P, G, false);        \
  } while (0)
#define LQ_STEP_P(P)                                  \
  do {                                                \
    if (plan.gdt == LOFTQ_BF16) LQ_STEP_G(P, __bf16); \
    else LQ_STEP_G(P, float);                         \
  } while (0)
  if (plan.pdt == LOFTQ_BF16) LQ_STEP_P(__bf16);
  else LQ_STEP_P(float);
#undef LQ_STEP_P
#undef LQ_STEP_G
#undef LQ_STEP
  return hipGetLastError();
}

}  // namespace loftq
