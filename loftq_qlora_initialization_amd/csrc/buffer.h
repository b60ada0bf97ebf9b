// Buffer resources: loads with a scalar base and 32-bit lane offsets, whose addresses cost no
// vector registers or instructions, and whose offsets at or past the resource's records touch no
// memory and give zeros, so that a loop needs no branch or select at its end.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace loftq {
namespace {

// `records` bytes from p (uniform; none where it is not positive; at most 2^31 - 1 are named).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t records) {
  const int n = records <= 0 ? 0 : (records < 0x7FFFFFFF ? static_cast<int>(records) : 0x7FFFFFFF);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, __builtin_amdgcn_readfirstlane(n), 0x00027000);
}
// Everything from p, or nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, bool any) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, __builtin_amdgcn_readfirstlane(any ? -1 : 0), 0x00027000);
}

}  // namespace
}  // namespace loftq
