// packed.h -- device-side lookup of packed sequences and request slots, and the
// limits of the heads' decay rates, shared by the SSD layer's kernels.
//
// Offsets, slots and positions are the caller's device memory, which the host
// cannot check: offsets are clamped to [0, total], a slot outside [0, nslots)
// means "no slot", a negative position counts as 0 and one past 2^62 as that, so a bad array gives
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

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// v of one lane (uniform) of the wave
__device__ __forceinline__ int64_t lane64(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// A run of 2^shift tokens of a sequence (its last one may be shorter).  Runs are numbered so that a wave
// finds the one of a number without a prefix sum over the lengths:
//   every run   run k of sequence s is (cu[s] >> shift) + s + k, all below (total >> shift) + nseq
//   full runs   that another one follows: (cu[s] >> shift) + k, all below total >> shift
// The numbers of one sequence end before the next one's begin; some name no run.
struct Run {
  int64_t s;            // sequence, -1: no run has this number
  int64_t start, stop;  // its tokens
  int64_t k;            // the run's number in it
};

// The run of a uniform number; whole waves.  Looks at 64 offsets at a time.
template <bool kFull>
__device__ __forceinline__ Run find_run(const Packed& p, int64_t number, int shift) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = p.nseq;
  while (n > 63) {
    const int64_t step = (n + 62) / 63, i = lo + lane * step;
    const bool in = lane * step < n && (seq_offset(p, i) >> shift) + (kFull ? 0 : i) <= number;
    const int c = __popcll(__ballot(in));
    if (c == 0) return Run{-1, 0, 0, 0};
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  // offsets lo .. lo + n, the last of them where the last sequence stops
  const int64_t v = seq_offset(p, lo + min((int64_t)lane, n));
  const int c = __popcll(__ballot(lane < n && (v >> shift) + (kFull ? 0 : lo + lane) <= number));
  if (c == 0) return Run{-1, 0, 0, 0};
  Run r;
  r.s = lo + c - 1;
  r.start = lane64(v, c - 1);
  r.stop = lane64(v, c);
  r.k = number - ((r.start >> shift) + (kFull ? 0 : r.s));
  // (k < 0 only where offsets fall)
  if (r.k < 0 || r.start + ((r.k + (kFull ? 1 : 0)) << shift) >= r.stop) r.s = -1;
  return r;
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
  return v < 0 ? 0 : min(v, (int64_t)1 << 62);   // room for the call's tokens
}

// A = -exp(A_log) in products with Delta is held at this, where exp(Delta A) is 0 for any Delta that is not: an
// infinite A would make Delta = 0 a NaN (a NaN stays one)
__device__ __forceinline__ float ssd_held(float rate) { return rate < -0x1p126f ? -0x1p126f : rate; }

// (exp(Delta A) - 1) / A is Delta where |Delta A| is below this, to 2^-26 of it; it is not divided
// there, since A may be too small a number to divide by
constexpr float kTinyStep = 0x1p-25f;

}  // namespace mscan
