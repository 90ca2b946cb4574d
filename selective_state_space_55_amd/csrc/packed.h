// packed.h -- device-side lookup of packed sequences and request slots, shared
// by the SSD layer's kernels.
//
// Offsets, slots and positions are the caller's device memory, which the host
// cannot check: offsets are clamped to [0, total], a slot outside [0, nslots)
// means "no slot" and a negative position counts as 0, so a bad array gives
// wrong results but no access out of bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

struct Packed {
  const int64_t* cu;         // (nseq + 1) offsets
  const int64_t* slots;      // (nseq) or null: no sequence has a slot
  const int64_t* positions;  // (nseq), tokens each sequence has behind it; null with slots
  int64_t nseq, total, nslots;
};

__device__ __forceinline__ int64_t seq_offset(const Packed& p, int64_t s) {
  const int64_t v = p.cu[s];
  return v < 0 ? 0 : v > p.total ? p.total : v;
}

// The last s in [0, nseq) with key(s) <= target, -1 if there is none; keys do
// not fall.  Whole wave, target uniform: a wave looks at 64 keys at a time.
template <typename Key>
__device__ __forceinline__ int64_t last_not_above(int64_t nseq, int64_t target, Key key) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = nseq;
  while (n > 64) {
    const int64_t step = (n + 63) / 64;
    const int64_t i = lo + lane * step;
    const int c = __popcll(__ballot(lane * step < n && key(i) <= target));
    if (c == 0) return -1;
    const int64_t off = (c - 1) * step;
    lo += off;
    n = min(step, n - off);
  }
  const int c = __popcll(__ballot(lane < n && key(lo + lane) <= target));
  return c == 0 ? -1 : lo + c - 1;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// the slot of sequence s, -1 if it has none
__device__ __forceinline__ int64_t seq_slot(const Packed& p, int64_t s) {
  if (!p.slots) return -1;
  const int64_t v = p.slots[s];
  return v < 0 || v >= p.nslots ? -1 : v;
}

// tokens behind sequence s
__device__ __forceinline__ int64_t seq_position(const Packed& p, int64_t s) {
  if (!p.slots) return 0;
  const int64_t v = p.positions[s];
  return v < 0 ? 0 : v;
}

}  // namespace mscan
