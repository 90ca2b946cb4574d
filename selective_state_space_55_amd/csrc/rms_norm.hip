// rms_norm.hip -- root-mean-square norm with the residual's addition on gfx950,
// with an io-typed or 8-bit (e4m3) output, and its gradient.
//
//   r = x + residual            (fp32; stored in the residual's type)
//   rstd = 1 / sqrt(mean(r^2) + eps),   y = r rstd weight
//
// 8-bit output: q = y / s rounded to e4m3 (OCP, 3 mantissa bits, largest 448),
// s = amax / 448 per row in fp32, or per 32 columns the smallest power of two
// with amax / s <= 448, stored as an e8m0 exponent byte (the block format that
// gfx950's scaled matrix instructions read).  s = 1 where all values are 0.
//
// Gradient, with xh = r rstd and g = dy weight:
//   dr = rstd (g - xh mean(g xh)) + d_residual,   dweight = sum_rows dy xh
//
// Both are streams (a row is read and written once, ~10 operations per
// element), so what bounds them is HBM; a row stays in registers between the
// sum of squares and its use.  W elements per access (8, or 1 for rows that are
// not 16-byte aligned), T lanes per row (a wave, so that the sum needs no LDS,
// or a 256-thread workgroup for long rows) and V accesses per lane.  32768 rows of 2560, bf16 to e4m3 with a
// scale per row: 119 - 126 us, 4.9 - 4.7 TB/s; the gradient of 32768 rows of 2048, bf16 with an fp32 residual: 198 us + 5
// for dweight, 5.3 TB/s (a copy of 1 GiB: 4.8 - 5.2); 16 rows: 5 us.
#include "internal.h"
#include "io.h"
#include "mfma.h"

#include <algorithm>

namespace mscan {
namespace {

constexpr int kThreads = 256;
constexpr int threads_of(int T) { return T > kThreads ? T : kThreads; }   // of a workgroup, with T lanes per row
constexpr float kFp8Max = 448.0f;

struct NArgs {
  const void* x;           // forward: x; backward: dy
  const void* res;         // forward: residual or null; backward: r
  const float* w;
  const float* rstd_in;    // backward
  const void* dres;        // backward: gradient of the residual stream, or null
  void* res_out;           // forward: r; backward: dresidual, or null
  void* y;                 // forward: y; backward: dx
  void* scales;
  float* rstd;             // forward output, or null
  float* part;             // backward: (gridDim.x, dim) partial dweight
  int64_t rows, dim;
  float eps;
  int res_f32;             // the residual's type is fp32 (else the io type)
  int out;                 // kNormIo, kNormRow8, kNormMx8
};

// total of a value over the wave, the same in every lane
__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_prefix_sum(v)), 63));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float v) {   // v >= 0
  return fmaxf(v, dpp_add_src<CTRL, ROWS>(v));
}

// largest of a value >= 0 over the wave, the same in every lane
__device__ __forceinline__ float wave_max(float v) {
  v = dpp_max<0x111, 0xf>(v);
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);
  v = dpp_max<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// over the T lanes of a row, T a wave or a whole workgroup; red: T / 64 floats, each call its own
template <int T, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* red) {
  v = kMax ? wave_max(v) : wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v = kMax ? fmaxf(v, red[i]) : v + red[i];
  }
  return v;
}

// largest over the lanes that hold one 32-column block: 4 lanes of 8 elements, or 32 of 1
template <int W>
__device__ __forceinline__ float block_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xf, 0xf, true)));   // lane ^ 1
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xf, 0xf, true)));   // lane ^ 2
  if constexpr (W == 1) {
    v = fmaxf(v, __shfl_xor(v, 4));
    v = fmaxf(v, __shfl_xor(v, 8));
    v = fmaxf(v, __shfl_xor(v, 16));
  }
  return v;
}

template <typename T, int W>
__device__ __forceinline__ void load_w(const void* p, int64_t i, float (&f)[W]) {
  const T* q = static_cast<const T*>(p) + i;
  if constexpr (W == 8)
    Io<T>::to_f32(Io<T>::load8(q), f);
  else
    f[0] = Io<T>::load1(q);
}

template <typename T, int W>
__device__ __forceinline__ void store_w(void* p, int64_t i, const float (&f)[W]) {
  T* q = static_cast<T*>(p) + i;
  if constexpr (W == 8)
    Io<T>::store8(q, Io<T>::from_f32(f));
  else
    Io<T>::store1(q, f[0]);
}

// load_w for data that the kernel reads once and no one soon after: 32768 rows of 2560 with e4m3 output take 123 us
// with these loads and 126 with plain ones, with bf16 output 129 and 135; of 2048 with an fp32 residual 155 and 147 (the
// gradient, whose stores are larger, 210 against 202)
template <typename T, int W>
__device__ __forceinline__ void load_once(const void* p, int64_t i, float (&f)[W]) {
  if constexpr (W == 8) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const T*>(p) + i);
    if constexpr (sizeof(T) == 2)
      Io<T>::to_f32(__builtin_bit_cast(typename Io<T>::V8, __builtin_nontemporal_load(q)), f);
    else
      Io<T>::to_f32(typename Io<T>::V8{__builtin_bit_cast(float4, __builtin_nontemporal_load(q)),
                                       __builtin_bit_cast(float4, __builtin_nontemporal_load(q + 1))}, f);
  } else {
    load_w<T, W>(p, i, f);
  }
}

template <int W>
__device__ __forceinline__ void store_fp8(void* p, int64_t i, const float (&f)[W]) {
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if constexpr (W == 8) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], b, true);
    *reinterpret_cast<uint2*>(q) = make_uint2((uint32_t)a, (uint32_t)b);
  } else {
    *q = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[0], 0, false);
  }
}

__device__ __forceinline__ float row_scale(float top) { return top > 0.0f ? fmaxf(top / kFp8Max, 0x1p-126f) : 1.0f; }

// exponent of a block's scale: top = 1.m 2^e, e - 8, one more where 1.m > 1.75 (448 = 1.75 2^8)
__device__ __forceinline__ int block_exp(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u == 0) return 0;
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(-127, min(127, k));
}

// A row whose mean square is outside of this range may have squares that fp32 does not hold (below it, squares that
// have lost bits matter): it is summed again, scaled by the power of two that row_exp gives.
__device__ __forceinline__ bool mean_square_ok(float ms) { return ms >= 0x1p-100f && ms < INFINITY; }

// k, so that the row's largest magnitude and sqrt(eps) are below 1 after a scaling by 2^-k and one of them is at least
// 1/2; 0 where there is nothing to scale (all 0, or an Inf, whose row is NaN)
__device__ __forceinline__ int row_exp(float top, float eps) {
  const float m = fmaxf(top, sqrtf(eps));
  return m > 0.0f && m < INFINITY ? __builtin_amdgcn_frexp_expf(m) : 0;
}

template <typename IoT, int W, int T, int V>
__global__ __launch_bounds__(threads_of(T)) void rms_norm_fwd_kernel(NArgs a) {
  __shared__ float red[4][16];
  const int64_t row = (int64_t)blockIdx.x * (threads_of(T) / T) + threadIdx.x / T;
  const int t = threadIdx.x % T;
  if (row >= a.rows) return;   // whole waves (T = 64) or no workgroup at all
  const int64_t base = row * a.dim;
  const int nvec = (int)(a.dim / W);
  float r[V][W];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * T + t < nvec) {
      load_once<IoT, W>(a.x, base + (int64_t)(v * T + t) * W, r[v]);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) r[v][j] = 0.0f;
    }
  }
  if (a.res) {
    float s[V][W];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t i = base + (int64_t)(v * T + t) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) s[v][j] = 0.0f;
      if (v * T + t < nvec) {
        if (a.res_f32)
          load_once<float, W>(a.res, i, s[v]);
        else
          load_once<IoT, W>(a.res, i, s[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t i = base + (int64_t)(v * T + t) * W;
#pragma unroll
      for (int j = 0; j < W; ++j) r[v][j] += s[v][j];
      if (v * T + t < nvec) {
        if (a.res_f32)
          store_w<float, W>(a.res_out, i, r[v]);
        else
          store_w<IoT, W>(a.res_out, i, r[v]);
      }
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < W; ++j) ss = fmaf(r[v][j], r[v][j], ss);
  ss = row_reduce<T, false>(ss, red[0]);
  float ms = ss / (float)a.dim + a.eps, top = 0.0f;
  int k = 0;   // r stands for r 2^-k, rstd for rstd 2^k
  if (!mean_square_ok(ms)) {   // all of the row's lanes
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) top = fmaxf(top, fabsf(r[v][j]));
    k = row_exp(row_reduce<T, true>(top, red[2]), a.eps);
    top = ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        r[v][j] = ldexpf(r[v][j], -k);
        ss = fmaf(r[v][j], r[v][j], ss);
      }
    ms = row_reduce<T, false>(ss, red[3]) / (float)a.dim + ldexpf(a.eps, -2 * k);
  }
  const float rstd = 1.0f / sqrtf(ms);
  if (a.rstd && t == 0) a.rstd[row] = ldexpf(rstd, -k);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int vec = v * T + t;
    if (vec < nvec) {
      float w[W];
      load_w<float, W>(a.w, (int64_t)vec * W, w);
#pragma unroll
      for (int j = 0; j < W; ++j) r[v][j] = r[v][j] * rstd * w[j];
      if (a.out == kNormIo) store_w<IoT, W>(a.y, base + (int64_t)vec * W, r[v]);
    }
    if (a.out == kNormRow8) {
#pragma unroll
      for (int j = 0; j < W; ++j) top = fmaxf(top, fabsf(r[v][j]));
    } else if (a.out == kNormMx8) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) m = fmaxf(m, fabsf(r[v][j]));
      const int b = block_exp(block_max<W>(m));
      if (vec < nvec) {
#pragma unroll
        for (int j = 0; j < W; ++j) r[v][j] = ldexpf(r[v][j], -b);
        store_fp8<W>(a.y, base + (int64_t)vec * W, r[v]);
        if (vec % (32 / W) == 0)
          static_cast<uint8_t*>(a.scales)[row * ((a.dim + 31) / 32) + vec / (32 / W)] = (uint8_t)(b + 127);
      }
    }
  }
  if (a.out == kNormRow8) {
    const float s = row_scale(row_reduce<T, true>(top, red[1]));
    const float inv = 1.0f / s;
    if (t == 0) static_cast<float*>(a.scales)[row] = s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v * T + t >= nvec) continue;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float q = r[v][j] * inv;
        r[v][j] = fmaf(fmaf(-q, s, r[v][j]), inv, q);   // r / s, correctly rounded but for rare last bits
      }
      store_fp8<W>(a.y, base + (int64_t)(v * T + t) * W, r[v]);
    }
  }
}

// Rows of any length, one workgroup each, read once for the sum of squares (twice more where it has to be scaled), once for
// the largest value (row scale) and once for the output.  x and the residual are read
// for the last time by the thread that then writes r there, so res_out may be res.
template <typename IoT>
__global__ __launch_bounds__(kThreads) void rms_norm_fwd_long_kernel(NArgs a) {
  __shared__ float red[4][4];
  const int64_t row = blockIdx.x, base = row * a.dim;
  const int t = threadIdx.x;
  auto value = [&](int64_t c) {
    float v = Io<IoT>::load1(static_cast<const IoT*>(a.x) + base + c);
    if (a.res)
      v += a.res_f32 ? static_cast<const float*>(a.res)[base + c] : Io<IoT>::load1(static_cast<const IoT*>(a.res) + base + c);
    return v;
  };
  float ss = 0.0f;
  for (int64_t c = t; c < a.dim; c += kThreads) {
    const float v = value(c);
    ss = fmaf(v, v, ss);
  }
  ss = row_reduce<kThreads, false>(ss, red[0]);
  float ms = ss / (float)a.dim + a.eps;
  int k = 0;
  if (!mean_square_ok(ms)) {
    float top = 0.0f;
    for (int64_t c = t; c < a.dim; c += kThreads) top = fmaxf(top, fabsf(value(c)));
    k = row_exp(row_reduce<kThreads, true>(top, red[2]), a.eps);
    ss = 0.0f;
    for (int64_t c = t; c < a.dim; c += kThreads) {
      const float v = ldexpf(value(c), -k);
      ss = fmaf(v, v, ss);
    }
    ms = row_reduce<kThreads, false>(ss, red[3]) / (float)a.dim + ldexpf(a.eps, -2 * k);
  }
  const float rstd = 1.0f / sqrtf(ms);
  if (a.rstd && t == 0) a.rstd[row] = ldexpf(rstd, -k);
  float s = 1.0f;
  if (a.out == kNormRow8) {
    float top = 0.0f;
    for (int64_t c = t; c < a.dim; c += kThreads) top = fmaxf(top, fabsf(ldexpf(value(c), -k) * rstd * a.w[c]));
    s = row_scale(row_reduce<kThreads, true>(top, red[1]));
    if (t == 0) static_cast<float*>(a.scales)[row] = s;
  }
  // whole waves run the same trips: a 32-column block is spread over 32 lanes
  for (int64_t c0 = 0; c0 < a.dim; c0 += kThreads) {
    const int64_t c = c0 + t;
    const bool in = c < a.dim;
    const float r = in ? value(c) : 0.0f;
    float y = in ? ldexpf(r, -k) * rstd * a.w[c] : 0.0f;
    if (a.out == kNormMx8) {
      const int b = block_exp(block_max<1>(fabsf(y)));
      y = ldexpf(y, -b);
      if (in && (c & 31) == 0) static_cast<uint8_t*>(a.scales)[row * ((a.dim + 31) / 32) + (c >> 5)] = (uint8_t)(b + 127);
    }
    if (!in) continue;
    if (a.res) {
      if (a.res_f32)
        static_cast<float*>(a.res_out)[base + c] = r;
      else
        Io<IoT>::store1(static_cast<IoT*>(a.res_out) + base + c, r);
    }
    const float out[1] = {a.out == kNormRow8 ? y / s : y};
    if (a.out == kNormIo)
      store_w<IoT, 1>(a.y, base + c, out);
    else
      store_fp8<1>(a.y, base + c, out);
  }
}

// Gradient.  A workgroup walks rows blockIdx.x, blockIdx.x + gridDim.x, ... (kThreads / T of
// them at a time) and keeps its columns' dweight sums in registers; the partial sums of the
// workgroups are added up by dweight_kernel in a fixed order.
template <typename IoT, int W, int T, int V>
__global__ __launch_bounds__(threads_of(T)) void rms_norm_bwd_kernel(NArgs a) {
  constexpr int kR = threads_of(T) / T;   // rows at a time
  __shared__ float red[2][16];
  __shared__ float sum[T == 64 ? V * 64 * W : 1];
  const int t = threadIdx.x % T;
  const int nvec = (int)(a.dim / W);
  float dw[V][W], w[V][W];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      dw[v][j] = 0.0f;
      w[v][j] = 0.0f;
    }
    if (v * T + t < nvec) load_w<float, W>(a.w, (int64_t)(v * T + t) * W, w[v]);
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kR + threadIdx.x / T; row < a.rows; row += (int64_t)gridDim.x * kR) {
    const int64_t base = row * a.dim;
    float g[V][W], r[V][W];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        g[v][j] = 0.0f;
        r[v][j] = 0.0f;
      }
      if (v * T + t < nvec) {
        const int64_t i = base + (int64_t)(v * T + t) * W;
        load_w<IoT, W>(a.x, i, g[v]);
        if (a.res_f32)
          load_w<float, W>(a.res, i, r[v]);
        else
          load_w<IoT, W>(a.res, i, r[v]);
      }
    }
    const float rstd = a.rstd_in[row];
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        r[v][j] *= rstd;   // xh
        dw[v][j] = fmaf(g[v][j], r[v][j], dw[v][j]);
        g[v][j] *= w[v][j];
        dot = fmaf(g[v][j], r[v][j], dot);
      }
    // two sets of LDS words in turn: a fast wave's next row does not overwrite what a slow one reads
    dot = row_reduce<T, false>(dot, red[turn]) / (float)a.dim;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v * T + t >= nvec) continue;
      const int64_t i = base + (int64_t)(v * T + t) * W;
      float d[W];
#pragma unroll
      for (int j = 0; j < W; ++j) d[j] = rstd * fmaf(-r[v][j], dot, g[v][j]);
      if (a.dres) {
        float s[W];
        if (a.res_f32)
          load_w<float, W>(a.dres, i, s);
        else
          load_w<IoT, W>(a.dres, i, s);
#pragma unroll
        for (int j = 0; j < W; ++j) d[j] += s[j];
      }
      if (a.y) store_w<IoT, W>(a.y, i, d);
      if (a.res_out) store_w<float, W>(a.res_out, i, d);
    }
  }
  if constexpr (T == 64) {   // the four waves' sums, one after another
    for (int k = 0; k < kR; ++k) {
      __syncthreads();
      if ((int)(threadIdx.x / T) != k) continue;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          float* s = sum + (v * T + t) * W + j;
          dw[v][j] += k ? *s : 0.0f;
          *s = dw[v][j];
        }
    }
  }
  if (T == 64 && threadIdx.x / T != kR - 1) return;   // the last wave holds the workgroup's sums
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * T + t < nvec) store_w<float, W>(a.part, (int64_t)blockIdx.x * a.dim + (int64_t)(v * T + t) * W, dw[v]);
}

// Rows of any length: the row's dot product and then dx, both from memory.
template <typename IoT>
__global__ __launch_bounds__(kThreads) void rms_norm_bwd_long_kernel(NArgs a) {
  __shared__ float red[4];
  const int64_t row = blockIdx.x, base = row * a.dim;
  const float rstd = a.rstd_in[row];
  auto at_r = [&](int64_t i) { return a.res_f32 ? static_cast<const float*>(a.res)[i] : Io<IoT>::load1(static_cast<const IoT*>(a.res) + i); };
  float dot = 0.0f;
  for (int64_t c = threadIdx.x; c < a.dim; c += kThreads)
    dot = fmaf(Io<IoT>::load1(static_cast<const IoT*>(a.x) + base + c) * a.w[c], at_r(base + c) * rstd, dot);
  dot = row_reduce<kThreads, false>(dot, red) / (float)a.dim;
  for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
    const int64_t i = base + c;
    const float g = Io<IoT>::load1(static_cast<const IoT*>(a.x) + i) * a.w[c];
    float d[1] = {rstd * fmaf(-(at_r(i) * rstd), dot, g)};
    if (a.dres)
      d[0] += a.res_f32 ? static_cast<const float*>(a.dres)[i] : Io<IoT>::load1(static_cast<const IoT*>(a.dres) + i);
    if (a.y) store_w<IoT, 1>(a.y, i, d);
    if (a.res_out) store_w<float, 1>(a.res_out, i, d);
  }
}

// Partial dweight of long rows: a thread per column, rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename IoT>
__global__ __launch_bounds__(kThreads) void dweight_long_kernel(NArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.dim) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const int64_t i = row * a.dim + c;
    const float r = a.res_f32 ? static_cast<const float*>(a.res)[i] : Io<IoT>::load1(static_cast<const IoT*>(a.res) + i);
    s = fmaf(Io<IoT>::load1(static_cast<const IoT*>(a.x) + i), r * a.rstd_in[row], s);
  }
  a.part[(int64_t)blockIdx.y * a.dim + c] = s;
}

// dweight[c] = sum of part[0 .. n)[c]: 16 columns a workgroup, 64 threads a column, so that a thread has few
// loads and all of them are in flight (512 parts x 2048 columns: 4.8 us; with four threads a column 39.7 us)
__global__ __launch_bounds__(1024) void dweight_kernel(const float* part, float* dw, int n, int64_t dim) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (int k = g; k < n; k += 64) s += part[(int64_t)k * dim + c];
  }
  red[g][col] = s;
  __syncthreads();
  for (int h = 32; h; h >>= 1) {
    if (g < h) red[g][col] += red[g + h][col];
    __syncthreads();
  }
  if (g == 0 && c < dim) dw[c] = red[0][col];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The shapes a row is run in.  Aligned rows: a wave per row while it holds the row in a few registers, then a
// workgroup (bf16 with an fp32 residual; forward, 16384 rows of 4096: 155 us against 171 with a wave of 8 accesses;
// gradient, which holds three rows' worth: 203 against 242, and at 2560 130 against 159 with 5 accesses).  Rows off 16-byte
// alignment go element by element, at most 8 per lane (8192 rows of 5001, forward: 150 us, with up to 32 per lane 323; of
// 5000, aligned, 97).
enum { kLong, kWave1, kWave2, kWave3, kWave4, kWave5, kGroup2, kGroup4, kGroup8, kOddWave, kOddGroup, kOddGroup2, kOddGroup4 };

int row_shape(int64_t dim, bool vec, bool backward) {
  if (vec) {
    if (dim <= 512) return kWave1;
    if (dim <= 1024) return kWave2;
    if (dim <= 1536) return kWave3;
    if (dim <= 2048) return kWave4;
    if (dim <= 2560 && !backward) return kWave5;
    if (dim <= 4096) return kGroup2;
    if (dim <= 8192) return kGroup4;
    return dim <= 16384 ? kGroup8 : kLong;
  }
  if (dim <= 512) return kOddWave;
  if (dim <= 2048) return kOddGroup;
  if (dim <= 4096) return kOddGroup2;
  return dim <= 8192 ? kOddGroup4 : kLong;
}

bool wave_per_row(int shape) { return (shape >= kWave1 && shape <= kWave5) || shape == kOddWave; }

#define MSCAN_NORM_SHAPE(SHAPE, KERNEL, GRID, W, T, V)                                                     \
  case SHAPE:                                                                                              \
    hipLaunchKernelGGL((KERNEL<IoT, W, T, V>), GRID, dim3(threads_of(T)), 0, s, a);                        \
    break;
#define MSCAN_NORM_SHAPES(KERNEL, GRID)                 \
  switch (shape) {                                      \
    MSCAN_NORM_SHAPE(kWave1, KERNEL, GRID, 8, 64, 1)    \
    MSCAN_NORM_SHAPE(kWave2, KERNEL, GRID, 8, 64, 2)    \
    MSCAN_NORM_SHAPE(kWave3, KERNEL, GRID, 8, 64, 3)    \
    MSCAN_NORM_SHAPE(kWave4, KERNEL, GRID, 8, 64, 4)    \
    MSCAN_NORM_SHAPE(kGroup2, KERNEL, GRID, 8, 256, 2)  \
    MSCAN_NORM_SHAPE(kGroup4, KERNEL, GRID, 8, 256, 4)  \
    MSCAN_NORM_SHAPE(kGroup8, KERNEL, GRID, 8, 256, 8)  \
    MSCAN_NORM_SHAPE(kOddWave, KERNEL, GRID, 1, 64, 8)  \
    MSCAN_NORM_SHAPE(kOddGroup, KERNEL, GRID, 1, 256, 8)   \
    MSCAN_NORM_SHAPE(kOddGroup2, KERNEL, GRID, 1, 512, 8)  \
    MSCAN_NORM_SHAPE(kOddGroup4, KERNEL, GRID, 1, 1024, 8) \
    default: return hipErrorInvalidValue;               \
  }

template <typename IoT>
hipError_t run_fwd(const NormArgs& p, hipStream_t s) {
  NArgs a{};
  a.x = p.x; a.res = p.residual; a.w = p.weight; a.res_out = p.residual_out; a.y = p.y; a.scales = p.scales;
  a.rstd = p.rstd; a.rows = p.rows; a.dim = p.dim; a.eps = p.eps; a.res_f32 = p.res_f32; a.out = p.out;
  const bool vec = p.dim % 8 == 0 && aligned16(p.x) && aligned16(p.residual) && aligned16(p.weight) &&
                   aligned16(p.residual_out) && aligned16(p.y);
  const int shape = row_shape(p.dim, vec, false);
  if (shape == kLong) {
    hipLaunchKernelGGL(rms_norm_fwd_long_kernel<IoT>, dim3((unsigned)p.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(wave_per_row(shape) ? (p.rows + 3) / 4 : p.rows));
  if (shape == kWave5)
    hipLaunchKernelGGL((rms_norm_fwd_kernel<IoT, 8, 64, 5>), grid, dim3(kThreads), 0, s, a);
  else
    MSCAN_NORM_SHAPES(rms_norm_fwd_kernel, grid)
  return hipGetLastError();
}

template <typename IoT>
hipError_t run_bwd(const NormArgs& p, hipStream_t s) {
  NArgs a{};
  a.x = p.x; a.res = p.residual; a.w = p.weight; a.rstd_in = p.rstd; a.dres = p.dres; a.res_out = p.residual_out;
  a.y = p.y; a.part = static_cast<float*>(p.workspace); a.rows = p.rows; a.dim = p.dim; a.res_f32 = p.res_f32;
  const bool vec = p.dim % 8 == 0 && aligned16(p.x) && aligned16(p.residual) && aligned16(p.weight) &&
                   aligned16(p.dres) && aligned16(p.residual_out) && aligned16(p.y);
  const int shape = row_shape(p.dim, vec, true);
  const int64_t parts = wave_per_row(shape) ? std::min<int64_t>((p.rows + 3) / 4, 512) : norm_bwd_parts(p.rows);
  if (p.rows == 0) {
    // no rows: dweight_kernel writes zeros
  } else if (shape == kLong) {
    hipLaunchKernelGGL(rms_norm_bwd_long_kernel<IoT>, dim3((unsigned)p.rows), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(dweight_long_kernel<IoT>, dim3((unsigned)((p.dim + kThreads - 1) / kThreads), (unsigned)parts),
                       dim3(kThreads), 0, s, a);
  } else {
    const dim3 grid((unsigned)parts);
    MSCAN_NORM_SHAPES(rms_norm_bwd_kernel, grid)
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(dweight_kernel, dim3((unsigned)((p.dim + 15) / 16)), dim3(1024), 0, s, a.part, p.dweight,
                     (int)parts, p.dim);
  return hipGetLastError();
}

}  // namespace

int64_t norm_bwd_parts(int64_t rows) { return std::min<int64_t>(rows, 1024); }

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream) {
  return a.io_bf16 ? run_fwd<uint16_t>(a, stream) : run_fwd<float>(a, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream) {
  return a.io_bf16 ? run_bwd<uint16_t>(a, stream) : run_bwd<float>(a, stream);
}

}  // namespace mscan
