// linear_attention_step.hip -- one token per request through linear attention with
// a fixed decay per head on gfx950, the requests' states in a pool by slot.  Per row
// and head, lam = exp(log_decay):
//
//   S[v, k] <- lam S[v, k] + x_v k_k       (fp32)
//   o[v] = c sum_k S[v, k] q_k
//
// What bounds it is the state: 8 K V bytes per (row, head) against a few hundred of everything else.  A workgroup
// takes (row, head, slice of NI x 256 / LN values): LN lanes hold a value's states as one float4 each, so a wave
// moves up to 1 KB of contiguous state per access, and all of a thread's state loads are issued before they are used.
//
// 256 rows of 40 heads of 128 x 128 (11 of them padding): 208 us, 6.2 TB/s: nothing is read twice, and the state passes by the
// caches.  One row of 16 heads: 3.7 us.
//
// The update adds the increment m S + x k, m = expm1(log_decay), so that its rounding error shrinks with the decay;
// where more than half decays it is lam S + x k.
#include "internal.h"
#include "io.h"

#include <algorithm>

namespace mscan {
namespace {

struct StArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  float* state;
  const int64_t* slots;
  const int64_t* positions;
  void* o;
  int64_t nslots, q_stride, k_stride, v_stride;
  int H, K, V, nslice;
  float scale;
};

// The next step comes a whole batch later: the state takes no place in the caches.
typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ float4 load_once(const float* p) {
  return __builtin_bit_cast(float4, __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p)));
}
__device__ __forceinline__ void store_once(float* p, float4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(f32x4, v), reinterpret_cast<f32x4*>(p));
}

template <typename IoT>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  const IoT* e = static_cast<const IoT*>(p) + i;
  return make_float4(Io<IoT>::load1(e), Io<IoT>::load1(e + 1), Io<IoT>::load1(e + 2), Io<IoT>::load1(e + 3));
}

template <typename IoT, int LN, int NI>
__global__ __launch_bounds__(256) void linear_attention_step_kernel(StArgs a) {
  constexpr int kRows = 256 / LN, PS = kRows * NI;   // values per pass, per workgroup
  const int t = threadIdx.x;
  const int per_row = a.H * a.nslice;
  const int64_t row = blockIdx.x / per_row;
  const int hs = blockIdx.x % per_row, h = hs / a.nslice;
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.nslots) return;   // no request in this row: nothing is read or written
  const bool started = a.positions[row] > 0;  // else a request's first token, whatever its slot holds
  const int k4 = (t % LN) * 4, v0 = (hs % a.nslice) * PS + t / LN;
  const bool in = k4 < a.K;
  float* st = a.state + ((slot * a.H + h) * a.V + v0) * a.K + k4;
  float4 s[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (started && in && v0 + i * kRows < a.V) s[i] = load_once(st + (int64_t)i * kRows * a.K);
  }
  float x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    x[i] = v0 + i * kRows < a.V
               ? Io<IoT>::load1(static_cast<const IoT*>(a.v) + row * a.v_stride + (int64_t)h * a.V + v0 + i * kRows) : 0.0f;
  float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
  if (in) {
    q = load4<IoT>(a.q, row * a.q_stride + (int64_t)h * a.K + k4);
    k = load4<IoT>(a.k, row * a.k_stride + (int64_t)h * a.K + k4);
  }
  const float ld = a.log_decay[h], m = expm1f(ld);
  const bool slow = m > -0.5f;
  const float f = slow ? m : expf(ld);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int v = v0 + i * kRows;
    float4 n;
    n.x = fmaf(f, s[i].x, x[i] * k.x) + (slow ? s[i].x : 0.0f);
    n.y = fmaf(f, s[i].y, x[i] * k.y) + (slow ? s[i].y : 0.0f);
    n.z = fmaf(f, s[i].z, x[i] * k.z) + (slow ? s[i].z : 0.0f);
    n.w = fmaf(f, s[i].w, x[i] * k.w) + (slow ? s[i].w : 0.0f);
    if (in && v < a.V) store_once(st + (int64_t)i * kRows * a.K, n);
    float y = fmaf(q.x, n.x, fmaf(q.y, n.y, fmaf(q.z, n.z, q.w * n.w)));
#pragma unroll
    for (int o = LN / 2; o; o >>= 1) y += __shfl_xor(y, o);
    if (t % LN == 0 && v < a.V)
      Io<IoT>::store1(static_cast<IoT*>(a.o) + row * (int64_t)a.H * a.V + (int64_t)h * a.V + v, a.scale * y);
  }
}

// lanes per value: float4 of its states, a power of two
int lanes_of(int K) {
  int n = 4;
  while (n * 4 < K) n *= 2;
  return n;
}

template <typename IoT, int LN>
hipError_t run(const StArgs& b, int64_t batch, int passes, hipStream_t s) {
  StArgs a = b;
  const int slice = passes * 256 / LN;
  a.nslice = (a.V + slice - 1) / slice;
  const dim3 grid((unsigned)(batch * a.H * a.nslice));
  if (passes == 8)
    hipLaunchKernelGGL((linear_attention_step_kernel<IoT, LN, 8>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((linear_attention_step_kernel<IoT, LN, 1>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename IoT>
hipError_t run_lanes(const StArgs& a, int64_t batch, int passes, hipStream_t s) {
  switch (lanes_of(a.K)) {
    case 4: return run<IoT, 4>(a, batch, passes, s);
    case 8: return run<IoT, 8>(a, batch, passes, s);
    case 16: return run<IoT, 16>(a, batch, passes, s);
    case 32: return run<IoT, 32>(a, batch, passes, s);
    case 64: return run<IoT, 64>(a, batch, passes, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// Values per workgroup: eight passes, or one where the launch would leave CUs idle.
int linear_attention_step_slice(int64_t batch, int64_t nheads, int64_t kdim, int64_t vdim) {
  const int pass = 256 / lanes_of((int)kdim);
  return batch * nheads * ((vdim + 8 * pass - 1) / (8 * pass)) < 512 ? pass : 8 * pass;
}

hipError_t launch_linear_attention_step(const LinearAttentionStepArgs& p, hipStream_t stream) {
  StArgs a{};
  a.q = p.q; a.k = p.k; a.v = p.v; a.log_decay = p.log_decay; a.state = p.state; a.slots = p.slots;
  a.positions = p.positions; a.o = p.o; a.nslots = p.nslots; a.q_stride = p.q_stride; a.k_stride = p.k_stride;
  a.v_stride = p.v_stride; a.H = (int)p.nheads; a.K = (int)p.kdim; a.V = (int)p.vdim; a.scale = p.scale;
  const int passes = linear_attention_step_slice(p.batch, p.nheads, p.kdim, p.vdim) * lanes_of(a.K) / 256;
  return p.io_bf16 ? run_lanes<uint16_t>(a, p.batch, passes, stream) : run_lanes<float>(a, p.batch, passes, stream);
}

}  // namespace mscan
