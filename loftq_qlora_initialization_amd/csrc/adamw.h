// The optimizer's step over many tensors: what its kernels and entry points share.
#pragma once

#include "internal.h"

namespace loftq {

constexpr int kStateBlock = 256;   // elements that share a scale with states in 8 bits: four a lane of a wave
constexpr int kChunk = 4096;       // elements of a workgroup, all of one tensor

// Numbers of a step that are the same for every element.
struct AdamScalars {
  double lr, bias1, root2;   // lr lr_factor; 1 - b1^t; 1 / sqrt(1 - b2^t)
  double clip;               // c; negative: the step changes nothing
};

struct AdamDecays {
  double b1, c1, b2, c2;   // c = 1 - b
  float eps;
};

// The table: tensors, then the chunks (tensor, number within it), then the steps' scratch.
struct AdamTable {
  loftq_adamw_tensor_t* tensors;
  int2* chunks;
  double* partials;      // kNormWorkgroups sums of squares
  AdamScalars* scalars;
  size_t bytes;
};
constexpr int kNormWorkgroups = 2048;

inline int64_t adam_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

inline AdamTable adam_table(void* base, int32_t count, int64_t chunks) {
  auto pad = [](size_t b) { return (b + 255) / 256 * 256; };
  AdamTable t{};
  char* p = static_cast<char*>(base);
  size_t used = 0;
  t.tensors = reinterpret_cast<loftq_adamw_tensor_t*>(p);
  used += pad(static_cast<size_t>(count) * sizeof(loftq_adamw_tensor_t));
  t.chunks = reinterpret_cast<int2*>(p + used);
  used += pad(static_cast<size_t>(chunks) * sizeof(int2));
  t.partials = reinterpret_cast<double*>(p + used);
  used += kNormWorkgroups * sizeof(double);
  t.scalars = reinterpret_cast<AdamScalars*>(p + used);
  used += pad(sizeof(AdamScalars));
  t.bytes = used;
  return t;
}

hipError_t launch_adamw_table(const loftq_adamw_tensor_t* tensors, int32_t count, const AdamTable& t, hipStream_t s);
hipError_t launch_adamw(const loftq_adamw_plan_t& plan, const AdamTable& t, const loftq_adamw_t& step, float* norm, hipStream_t s);

}  // namespace loftq
