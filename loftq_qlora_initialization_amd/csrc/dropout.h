// The dropout mask shared by every kernel that drops elements: a function of
// (seed, offset, element index), so it is formed again wherever it is needed and
// never stored.
//
// Generator: SplitMix64 (Steele, Lea and Flood, "Fast splittable pseudorandom number
// generators", OOPSLA 2014), the sketch's generator: output w of the sequence started
// at s is mix(s + (w + 1) gamma).  A call's key is output offset + *step of the
// sequence started at seed; element i of the row-major flattening takes 16 bits, lane
// i % 4 (from the low end) of output i / 4 of the sequence started at key, and stays
// where they are at least thr = round(2^16 p).  One 64-bit output serves four
// elements: 10 32-bit multiplies and about 20 other operations for four.  The kept
// share is exactly 1 - thr / 2^16, so the scale 2^16 / (2^16 - thr) leaves the mean as
// it was.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace loftq {

struct DropArg {
  uint64_t seed, offset;
  const uint64_t* step;   // device, or null
  uint32_t thr;           // 0: nothing is dropped
  float scale;            // 2^16 / (2^16 - thr), 0 when everything is dropped
};

namespace {

constexpr uint64_t kMixGamma = 0x9E3779B97F4A7C15ull;

__device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

__device__ __forceinline__ uint64_t drop_key(const DropArg& d) {
  const uint64_t at = d.offset + (d.step != nullptr ? *d.step : 0);
  return mix64(d.seed + (at + 1) * kMixGamma);
}

// the 64 bits of elements 4 w .. 4 w + 3
__device__ __forceinline__ uint64_t drop_word(uint64_t key, uint64_t w) { return mix64(key + (w + 1) * kMixGamma); }

__device__ __forceinline__ bool drop_keeps(uint64_t word, int lane, uint32_t thr) {
  return (static_cast<uint32_t>(word >> (16 * lane)) & 0xFFFFu) >= thr;
}

// Two bf16 values of a packed word, elements `lane` and `lane` + 1 of the mask word: a dropped one becomes 0.
__device__ __forceinline__ uint32_t drop_pair(uint32_t v, uint64_t word, int lane, uint32_t thr) {
  const uint32_t lo = drop_keeps(word, lane, thr) ? 0x0000FFFFu : 0u;
  const uint32_t hi = drop_keeps(word, lane + 1, thr) ? 0xFFFF0000u : 0u;
  return v & (lo | hi);
}

}  // namespace
}  // namespace loftq
