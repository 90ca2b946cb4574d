// ssd_step.hip -- one token per request through the SSD layer's core on gfx950:
// the short convolution + SiLU of the token's x | B | C channels, the state
// update, the readout, the D skip and the gate, in one launch, the requests'
// inputs and states in pools by slot.  Per row, head h (group g), channel p:
//
//   u = SiLU(bias + sum_k w[k] v[pos - (K - 1) + k])          (x, B, C; fp32, not rounded)
//   a = exp(Delta A_h),  wt = (a - 1) / A_h  (Delta with the Euler input term)
//   h[p, n] <- a h[p, n] + wt x[p] B[n]
//   y[p] = (sum_n C[n] h[p, n] + D x[p]) SiLU(z[p])
//
// What bounds it is the fp32 state: 8 P N bytes per (row, head) against ~1 KB of
// everything else.  A workgroup takes (row, head, slice of kNI x 256 / (N / 4)
// channels): N / 4 lanes hold a channel's states as one float4 each, so a wave
// moves 1 KB of contiguous state per access, and all of a thread's state loads
// are issued before the convolution's.  B and C are formed by every workgroup of
// a row's group (2 N channels of K rows each, from L2).  The state's input row
// goes to ring row pos mod K, which no workgroup of the launch reads (they look
// back K - 1 rows): x's channels are written by their own workgroup, B's and C's
// by the first one of the group.
//
// 256 rows of 80 heads x 64 x 128, bf16: 248 us, 5.5 TB/s; one row 6 us, a chain of latencies (slot, position,
// ring and taps, the sum over a channel's states).
//
// The update adds the increment m h + wt x B, m = expm1(Delta A), so that its
// rounding error shrinks with Delta |A|.
#include "internal.h"
#include "io.h"
#include "packed.h"

#include <algorithm>

namespace mscan {
namespace {

struct StArgs {
  const void* xbc;
  const void* dt;
  const float* A_log;
  const float* cw;
  const float* cb;
  void* ring;
  float* state;
  const int64_t* slots;
  const int64_t* positions;
  const float* D;
  const void* z;
  const float* dt_bias;
  void* y;
  int64_t nslots, xbc_stride, dt_stride, z_stride, width;
  int H, P, G, nslice;
  int softplus, euler;
};

// A step reads and writes each state once and the next step comes a whole batch later: without a place in the
// caches 256 rows of 80 heads x 64 x 128 take 248 us, with one 267
typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ float4 load_once(const float* p) {
  return __builtin_bit_cast(float4, __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p)));
}
__device__ __forceinline__ void store_once(float* p, float4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(f32x4, v), reinterpret_cast<f32x4*>(p));
}

template <typename IoT, int N, int NI, int K>
__global__ __launch_bounds__(256) void ssd_step_kernel(StArgs a) {
  constexpr int LN = N / 4;          // lanes per channel
  constexpr int kRows = 256 / LN;    // channels per pass
  constexpr int PS = kRows * NI;     // channels per workgroup
  __shared__ float ub[N], uc[N], ux[PS], yp[PS];
  lds_poison(ub, sizeof(ub));
  lds_poison(uc, sizeof(uc));
  lds_poison(ux, sizeof(ux));
  lds_poison(yp, sizeof(yp));
  const int t = threadIdx.x;
  const int per_row = a.H * a.nslice;
  const int64_t row = blockIdx.x / per_row;
  const int hs = blockIdx.x % per_row;
  const int h = hs / a.nslice, p0 = (hs % a.nslice) * PS;
  const int g = h / (a.H / a.G);
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.nslots) return;   // no request in this row: nothing is read or written
  const int64_t pos = max(a.positions[row], (int64_t)0);

  const int n4 = (t % LN) * 4, pr = t / LN;
  float* st = a.state + ((slot * a.H + h) * a.P + p0 + pr) * N + n4;
  float4 s[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) s[i] = load_once(st + (int64_t)i * kRows * N);

  // the convolution of 2 N + PS channels
  const IoT* xr = static_cast<const IoT*>(a.xbc) + row * a.xbc_stride;
  IoT* ring = static_cast<IoT*>(a.ring) + slot * K * a.width;
  const int64_t inner = (int64_t)a.H * a.P;
  const int64_t now = pos % K;
  for (int i = t; i < 2 * N + PS; i += 256) {
    const int64_t c = i < N ? inner + g * N + i
                    : i < 2 * N ? inner + (int64_t)a.G * N + g * N + (i - N) : (int64_t)h * a.P + p0 + (i - 2 * N);
    const IoT raw = xr[c];
    float acc = a.cb ? a.cb[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      const int back = K - 1 - k;
      const float v = pos >= back ? Io<IoT>::load1(ring + ((pos - back) % K) * a.width + c) : 0.0f;
      acc = fmaf(a.cw[c * K + k], v, acc);
    }
    acc = fmaf(a.cw[c * K + K - 1], Io<IoT>::load1(&raw), acc);
    acc = acc / (1.0f + expf(-acc));
    if (i < N) ub[i] = acc;
    else if (i < 2 * N) uc[i - N] = acc;
    else ux[i - 2 * N] = acc;
    if (i >= 2 * N || hs == g * (a.H / a.G) * a.nslice) ring[now * a.width + c] = raw;
  }
  const float rate = -expf(a.A_log[h]), A = ssd_held(rate);
  const float dr = Io<IoT>::load1(static_cast<const IoT*>(a.dt) + row * a.dt_stride + h) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
  const float delta = a.softplus ? softplus_log2e(dr) * 0.6931471805599453f : dr;
  const float m = expm1f(delta * A);
  const float wt = a.euler || fabsf(delta * A) < kTinyStep ? delta : m / rate;
  __syncthreads();

  const float4 b = *reinterpret_cast<const float4*>(ub + n4), cc = *reinterpret_cast<const float4*>(uc + n4);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float4 v = pos > 0 ? s[i] : make_float4(0.f, 0.f, 0.f, 0.f);   // a request's first token
    const float wx = wt * ux[i * kRows + pr];
    v.x += fmaf(m, v.x, wx * b.x);
    v.y += fmaf(m, v.y, wx * b.y);
    v.z += fmaf(m, v.z, wx * b.z);
    v.w += fmaf(m, v.w, wx * b.w);
    store_once(st + (int64_t)i * kRows * N, v);
    float y = fmaf(cc.x, v.x, fmaf(cc.y, v.y, fmaf(cc.z, v.z, cc.w * v.w)));
#pragma unroll
    for (int o = LN / 2; o; o >>= 1) y += __shfl_xor(y, o);
    if (t % LN == 0) yp[i * kRows + pr] = y;
  }
  __syncthreads();
  for (int i = t; i < PS; i += 256) {
    float y = fmaf(a.D ? a.D[h] : 0.0f, ux[i], yp[i]);
    const int64_t c = (int64_t)h * a.P + p0 + i;
    if (a.z) {
      const float z = Io<IoT>::load1(static_cast<const IoT*>(a.z) + row * a.z_stride + c);
      y *= z / (1.0f + expf(-z));
    }
    Io<IoT>::store1(static_cast<IoT*>(a.y) + row * inner + c, y);
  }
}

template <typename IoT, int N, int NI>
hipError_t run_k(const StArgs& a, int K, dim3 grid, hipStream_t s) {
  switch (K) {
    case 2: hipLaunchKernelGGL((ssd_step_kernel<IoT, N, NI, 2>), grid, dim3(256), 0, s, a); break;
    case 3: hipLaunchKernelGGL((ssd_step_kernel<IoT, N, NI, 3>), grid, dim3(256), 0, s, a); break;
    case 4: hipLaunchKernelGGL((ssd_step_kernel<IoT, N, NI, 4>), grid, dim3(256), 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <typename IoT>
hipError_t run(const SsdStepArgs& p, hipStream_t s) {
  StArgs a{};
  a.xbc = p.xbc; a.dt = p.dt; a.A_log = p.A_log; a.cw = p.conv_weight; a.cb = p.conv_bias; a.ring = p.conv_state;
  a.state = p.state; a.slots = p.slots; a.positions = p.positions; a.D = p.D; a.z = p.z; a.dt_bias = p.dt_bias; a.y = p.y;
  a.nslots = p.nslots; a.xbc_stride = p.xbc_stride; a.dt_stride = p.dt_stride; a.z_stride = p.z_stride;
  a.H = p.nheads; a.P = p.headdim; a.G = p.ngroups; a.softplus = p.softplus; a.euler = p.euler;
  a.width = (int64_t)p.nheads * p.headdim + 2 * (int64_t)p.ngroups * p.dstate;
  const int ps = ssd_step_slice(p);
  a.nslice = p.headdim / ps;
  const dim3 grid((unsigned)(p.batch * p.nheads * a.nslice));
  const int ni = ps * p.dstate / 1024;   // passes of 1024 / N channels
  if (p.dstate == 128) {
    if (ni == 8) return run_k<IoT, 128, 8>(a, p.K, grid, s);
    if (ni == 4) return run_k<IoT, 128, 4>(a, p.K, grid, s);
    return run_k<IoT, 128, 1>(a, p.K, grid, s);
  }
  if (ni == 4) return run_k<IoT, 64, 4>(a, p.K, grid, s);
  if (ni == 2) return run_k<IoT, 64, 2>(a, p.K, grid, s);
  return run_k<IoT, 64, 1>(a, p.K, grid, s);
}

}  // namespace

// 64 channels per workgroup, 32 where the head dim is an odd multiple of 32, and the
// fewest that fill one pass where the launch would leave CUs idle
int ssd_step_slice(const SsdStepArgs& a) {
  const int ps = a.headdim % 64 == 0 ? 64 : 32;
  return a.batch * a.nheads * (a.headdim / ps) < 512 ? 1024 / a.dstate : ps;
}

hipError_t launch_ssd_step(const SsdStepArgs& a, hipStream_t stream) {
  return a.io_bf16 ? run<uint16_t>(a, stream) : run<float>(a, stream);
}

}  // namespace mscan
