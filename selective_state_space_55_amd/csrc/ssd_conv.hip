// ssd_conv.hip -- the short causal convolution + SiLU in front of the SSD, over
// packed prompts, token-major (a token's x | B | C channels contiguous, as the
// in-projection leaves them).
//
//   u[t, c] = SiLU(bias[c] + sum_{k<K} w[c, k] v[p - (K - 1) + k]),  p = the token's position
//
// v[q] is the sequence's input at position q: a row of x for tokens of this
// call, ring row q mod K of the sequence's slot for the tokens before it, 0 for
// q < 0.  A ring of K rows (one more than the K - 1 a token looks back) lets the
// single-token kernel write a new row that no workgroup of that launch reads, and
// nothing is ever shifted.
//
// A stream (x read once, u written once), bound by HBM.  A wave takes a run of
// up to kRun tokens of one sequence, a lane W channels of it (8: one 16-byte
// access, or 1 where rows are not 16-byte aligned), so its K - 1 previous inputs
// stay in registers.  Runs are counted from each sequence's start (run k of
// sequence s has number cu[s] / kRun + s + k; see packed.h), so only a
// sequence's first run looks at the ring: it reads the rows behind it and then
// writes the new ones, and no other wave has to be waited for.  28 sequences of 32768 tokens, 4352 channels in
// bf16: 119 - 137 us, 4.8 - 4.2 TB/s (a copy of 1 GiB: 5.2 - 4.8); with tokens 4353 elements apart, which take 2-byte
// accesses, 144 against 119 on the same card; in fp32 224 us, 5.1 TB/s.  333 tokens of 5 sequences, 1792 channels:
// 9.5 us, the latency of its chain (offsets, slot, ring, taps).
#include "internal.h"
#include "io.h"
#include "packed.h"

#include <algorithm>

namespace mscan {
namespace {

// tokens a wave walks: 32768 x 4352 bf16 takes 129 us with 8, 190 with 4 (taps and history are read too
// often for them) and 209 with 16 (twice the registers, half the waves)
constexpr int kRunShift = 3, kRun = 1 << kRunShift;

struct CArgs {
  Packed seq;
  const void* x;
  const float* w;
  const float* bias;
  void* ring;      // (nslots, K, width) or null
  void* u;
  int64_t width, xstride;
  int silu;
  unsigned ngroups;   // groups of 64 lanes of channels
};

// W elements as they lie in memory
template <typename IoT, int W>
struct Raw {
  typename Io<IoT>::V8 v;
  __device__ __forceinline__ void load(const IoT* p) { v = Io<IoT>::load8(p); }
  __device__ __forceinline__ void zero() { v = Io<IoT>::zero(); }
  __device__ __forceinline__ void f32(float (&f)[W]) const { Io<IoT>::to_f32(v, f); }
};
template <typename IoT>
struct Raw<IoT, 1> {
  IoT v;
  __device__ __forceinline__ void load(const IoT* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = IoT(0); }
  __device__ __forceinline__ void f32(float (&f)[1]) const { f[0] = Io<IoT>::load1(&v); }
};

template <typename IoT, int W, int K>
__global__ __launch_bounds__(256) void ssd_conv_kernel(CArgs a) {
  const int lane = threadIdx.x & 63;
  const Packed& q = a.seq;
  const Run r = find_run<false>(q, uniform64((int64_t)(blockIdx.x / a.ngroups) * 4 + (threadIdx.x >> 6)), kRunShift);
  if (r.s < 0) return;   // whole waves
  const int64_t s = r.s, start = r.start, end = r.stop, k0 = r.k, t0 = start + k0 * kRun;
  const int64_t c = ((int64_t)(blockIdx.x % a.ngroups) * 64 + lane) * W;
  if (c >= a.width) return;
  const IoT* x = static_cast<const IoT*>(a.x) + c;
  IoT* u = static_cast<IoT*>(a.u) + c;
  IoT* ring = static_cast<IoT*>(a.ring) + c;

  // v[0 .. K-2]: the inputs behind the run, v[K-1 ..]: the run's own, all loads before the first use
  Raw<IoT, W> v[K - 1 + kRun];
  float w[W][K], b[W];
#pragma unroll
  for (int i = 0; i < kRun; ++i) v[K - 1 + i].load(x + min(t0 + i, end - 1) * a.xstride);
  const int64_t slot = k0 ? -1 : seq_slot(q, s);
  const int64_t pos = slot < 0 ? 0 : seq_position(q, s);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int64_t p = pos - (K - 1) + i;
    v[i].zero();
    if (k0)
      v[i].load(x + (t0 - (K - 1) + i) * a.xstride);
    else if (slot >= 0 && p >= 0)
      v[i].load(ring + (slot * K + p % K) * a.width);
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[j][k] = a.w[(c + j) * K + k];
    b[j] = a.bias ? a.bias[c + j] : 0.0f;
  }
  if (slot >= 0) {   // the sequence's first run: the rows of its last tokens
    const int64_t n = min(end - start, (int64_t)(K - 1));
    for (int64_t i = 1; i <= n; ++i) {
      IoT* to = ring + (slot * K + (pos + end - start - i) % K) * a.width;
      const IoT* from = x + (end - i) * a.xstride;
#pragma unroll
      for (int j = 0; j < W; ++j) to[j] = from[j];
    }
  }
  const int n = (int)min((int64_t)kRun, end - t0);
  float f[K][W];   // the last K inputs, in turn
#pragma unroll
  for (int i = 0; i < K - 1; ++i) v[i].f32(f[i]);
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    if (i >= n) break;
    v[i + K - 1].f32(f[(i + K - 1) % K]);
    float out[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float acc = b[j];
#pragma unroll
      for (int k = 0; k < K; ++k) acc = fmaf(w[j][k], f[(i + k) % K][j], acc);
      out[j] = a.silu ? silu(acc) : acc;
    }
    if constexpr (W == 8)
      Io<IoT>::store8(u + (t0 + i) * a.width, Io<IoT>::from_f32(out));
    else
      Io<IoT>::store1(u + (t0 + i) * a.width, out[0]);
  }
}

template <typename IoT, int W>
hipError_t run(CArgs a, int K, hipStream_t s) {
  a.ngroups = (unsigned)((a.width + 64 * W - 1) / (64 * W));
  // channel groups of a run next to each other, so that what is read at a time is whole rows (136 us the other way round)
  const dim3 grid((unsigned)((ssd_conv_runs(a.seq.nseq, a.seq.total) + 3) / 4 * a.ngroups));
  switch (K) {
    case 2: hipLaunchKernelGGL((ssd_conv_kernel<IoT, W, 2>), grid, dim3(256), 0, s, a); break;
    case 3: hipLaunchKernelGGL((ssd_conv_kernel<IoT, W, 3>), grid, dim3(256), 0, s, a); break;
    case 4: hipLaunchKernelGGL((ssd_conv_kernel<IoT, W, 4>), grid, dim3(256), 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

// the run numbers end below total / kRun + nseq
int64_t ssd_conv_runs(int64_t nseq, int64_t total) { return total / kRun + nseq; }

hipError_t launch_ssd_conv(const SsdConvArgs& p, hipStream_t stream) {
  CArgs a{};
  a.seq.cu = p.cu; a.seq.slots = p.slots; a.seq.positions = p.positions;
  a.seq.nseq = p.nseq; a.seq.total = p.total; a.seq.nslots = p.nslots;
  a.x = p.x; a.w = p.weight; a.bias = p.bias; a.ring = p.conv_state; a.u = p.u;
  a.width = p.width; a.xstride = p.x_stride; a.silu = p.silu;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.u) |
                        reinterpret_cast<uintptr_t>(p.conv_state);
  const int64_t e = p.io_bf16 ? 2 : 4;
  const bool vec = p.width % 8 == 0 && (mis & 15) == 0 && (p.x_stride * e) % 16 == 0;
  if (p.io_bf16) return vec ? run<uint16_t, 8>(a, p.K, stream) : run<uint16_t, 1>(a, p.K, stream);
  return vec ? run<float, 8>(a, p.K, stream) : run<float, 1>(a, p.K, stream);
}

}  // namespace mscan
