// The sequence of a packed row, found by a wavefront together (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace {

// The last of n_seqs sequences for which begun(s) holds (0 if there is none; it holds up to some sequence): 64 are looked
// at in one load, so up to 64 sequences take one round trip to memory and up to 4096 two.  All lanes give the same answer.
template <class F>
__device__ __forceinline__ uint32_t last_begun(uint32_t n_seqs, uint32_t lane, F begun) {
  uint32_t lo = 0, span = n_seqs;
  while (span > 1) {
    const uint32_t step = (span + 63) / 64, i = lane * step;
    const bool before = i < span && begun(lo + i);
    const uint32_t k = (uint32_t)max(__builtin_popcountll(__ballot(before)), 1) - 1;
    lo += k * step;
    span = min(step, span - k * step);
  }
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)lo);
}

// The sequence of row t: the last with starts[s] <= t.
__device__ __forceinline__ uint32_t seq_at(const int32_t* starts, uint32_t n_seqs, int32_t t, uint32_t lane) {
  return last_begun(n_seqs, lane, [&](uint32_t s) { return starts[s] <= t; });
}

}  // namespace
