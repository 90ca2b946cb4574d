// group_norm.hip -- norm of groups of a row's channels with an activation, and its
// gradient, on gfx950.  For each row and each group of `width` consecutive channels
//
//   n = (x - mean) / sqrt(var + eps) weight + bias      (without centring mean = 0, var = mean(x^2))
//   y = n,  SiLU(n)  or  n SiLU(z)
//
// Gradient, with xh = (x - mean) rstd, s(.) the sigmoid and dn = dy, dy SiLU'(n) or dy SiLU(z):
//
//   g = dn weight,   dx = rstd (g - mean(g) - xh mean(g xh))     (without centring no mean(g))
//   dz = dy n SiLU'(z),   dweight = sum over rows of dn xh,   dbias = sum over rows of dn
//
// Streams: each array is read or written once, ~15 operations per element, so what bounds them is HBM.  A group stays
// in registers, in T lanes of V accesses of W elements.  Groups of 128 in bf16: 32768 x 4096 with a gate 157 us, 5.1 TB/s;
// its gradient over 16384 x 4096, gate, weight and bias, 135 us and 5 for the sums, 5.0 TB/s; 16 x 2048 3.3 us.
#include "internal.h"
#include "io.h"
#include "mfma.h"

#include <algorithm>

namespace mscan {
namespace {

constexpr int threads_of(int T) { return T > 256 ? T : 256; }

struct GArgs {
  const void* dy;      // gradient only
  const void* x;
  const void* z;       // or null
  const float* w;      // or null
  const float* b;      // or null
  void* y;             // forward: y; gradient: dx
  void* dz;            // written iff z
  float* part;         // gradient: (parts, 2, dim) sums for dweight and dbias
  int64_t rows, z_stride;
  int G, width;
  int center, silu;
  int want_w, want_b;
  float eps;
};

// sum (or the largest) over the T lanes of a group, the same in each; red: T / 64 floats of its own each call
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

template <bool kMax>
__device__ __forceinline__ float join(float a, float b) { return kMax ? fmaxf(a, b) : a + b; }

template <int T, bool kMax = false>
__device__ __forceinline__ float group_reduce(float v, float* red) {
  v = join<kMax>(v, dpp_move<0xB1>(v));    // lane ^ 1
  v = join<kMax>(v, dpp_move<0x4E>(v));    // lane ^ 2
  v = join<kMax>(v, dpp_move<0x141>(v));   // mirrored in 8: the other four's
  if constexpr (T >= 16) v = join<kMax>(v, dpp_move<0x140>(v));   // mirrored in 16: the other eight's
  if constexpr (T >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = join<kMax>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (T >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = join<kMax>(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v = join<kMax>(v, red[i]);
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

__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * 1.4426950408889634f));
}

constexpr int kReds = 9;   // reductions of a group, at most

// x becomes (x - mean) rstd; returns rstd.  The mean is taken twice, the second time of what the first leaves, so that
// a group of nearly equal values keeps its differences.  Where the squares leave fp32's range (below it, where those that
// have lost bits matter), or nothing but the mean's rounding may be left, the group is taken again, scaled by a power of
// two, and one of equal values as such.
template <int W, int T, int V>
__device__ __forceinline__ float normalise(const GArgs& a, float (&x)[V][W], int t, float (*red)[16]) {
  const int nvec = a.width / W;
  const float inv = 1.0f / (float)a.width;
  float raw[V][W], mean = 0.0f, md = 0.0f, ms = 0.0f, eps = a.eps;
  int k = 0;
  auto moments = [&](int at) {
    mean = 0.0f;
    if (a.center) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) mean += x[v][j];
      mean = group_reduce<T>(mean, red[at]) * inv;
    }
    float s = 0.0f, ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        x[v][j] = v * T + t < nvec ? x[v][j] - mean : 0.0f;
        s += x[v][j];
        ss = fmaf(x[v][j], x[v][j], ss);
      }
    md = a.center ? group_reduce<T>(s, red[at + 1]) * inv : 0.0f;
    ms = fmaf(-md, md, group_reduce<T>(ss, red[at + 2]) * inv);
    ms = ms < 0.0f ? 0.0f : ms;   // (a NaN stays one)
  };
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < W; ++j) raw[v][j] = x[v][j];
  moments(0);
  if (!(ms + eps >= fmaxf(0x1p-100f, 0x1p-40f * mean * mean) && ms < 0x1p126f)) {   // all of the group's lanes
    float up = -INFINITY, down = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        up = v * T + t < nvec ? fmaxf(up, raw[v][j]) : up;
        down = v * T + t < nvec ? fmaxf(down, -raw[v][j]) : down;
      }
    up = group_reduce<T, true>(up, red[3]);
    down = group_reduce<T, true>(down, red[7]);
    const float top = fmaxf(fmaxf(up, down), sqrtf(eps));
    const bool equal = a.center && up == -down;
    k = top > 0.0f && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] = equal && raw[v][j] == up ? 0.0f : ldexpf(raw[v][j], -k);   // (not a NaN)
    if (eps > 0.0f) eps = fmaxf(ldexpf(eps, -2 * k), 0x1p-126f);   // (not 0: equal values give 0)
    moments(4);
  }
  const float rstd = 1.0f / sqrtf(ms + eps);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < W; ++j) x[v][j] = (x[v][j] - md) * rstd;
  return ldexpf(rstd, -k);
}

template <typename IoT, int W, int T, int V>
__global__ __launch_bounds__(threads_of(T)) void group_norm_fwd_kernel(GArgs a) {
  __shared__ float red[kReds][16];
  const int64_t unit = (int64_t)blockIdx.x * (threads_of(T) / T) + threadIdx.x / T;
  const int t = threadIdx.x % T, nvec = a.width / W;
  const bool some = unit < a.rows * a.G;   // (always, where a group takes a workgroup)
  const int64_t row = some ? (int64_t)((uint32_t)unit / (uint32_t)a.G) : 0;
  const int g = some ? (int)(unit - row * a.G) : 0;
  const int64_t base = unit * a.width;
  float x[V][W], z[V][W];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + t) * W;
    const bool in = some && v * T + t < nvec;
#pragma unroll
    for (int j = 0; j < W; ++j) x[v][j] = z[v][j] = 0.0f;
    if (in) load_w<IoT, W>(a.x, base + c, x[v]);
    if (in && a.z) load_w<IoT, W>(a.z, row * a.z_stride + (int64_t)g * a.width + c, z[v]);
  }
  normalise<W, T, V>(a, x, t, red);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!(some && v * T + t < nvec)) continue;
    const int c = (v * T + t) * W;
    if (a.w) {
      float w[W];
      load_w<float, W>(a.w, (int64_t)g * a.width + c, w);
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] *= w[j];
    }
    if (a.b) {
      float b[W];
      load_w<float, W>(a.b, (int64_t)g * a.width + c, b);
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] += b[j];
    }
    if (a.z) {
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] *= z[v][j] * sigmoid(z[v][j]);
    } else if (a.silu) {
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] *= sigmoid(x[v][j]);
    }
    store_w<IoT, W>(a.y, base + c, x[v]);
  }
}

// Gradient.  A wave takes `gw` neighbouring groups of `rw` rows at a time (a workgroup one group, where that takes all
// of it), the same groups all along, so that a lane's columns, and with them the sums for dweight and dbias, stay.
template <typename IoT, int W, int T, int V>
__global__ __launch_bounds__(threads_of(T)) void group_norm_bwd_kernel(GArgs a, int gw, int cblocks) {
  constexpr int kWaves = T > 64 ? 1 : 4;   // that walk rows of their own
  __shared__ float red[2][kReds + 2][16];
  __shared__ float sums[T > 64 ? 1 : 256][W];
  const int t = threadIdx.x % T, nvec = a.width / W;
  const int sub = T > 64 ? 0 : (threadIdx.x & 63) / T, rw = T > 64 ? 1 : 64 / T / gw;
  const int cb = blockIdx.x % cblocks;
  const int64_t rb = blockIdx.x / cblocks, rblocks = gridDim.x / cblocks;
  const int g = cb * gw + sub % gw;
  const bool lane_in = g < a.G && sub / gw < rw;
  const int64_t step = rblocks * kWaves * rw;
  float w[V][W], b[V][W], dw[V][W], db[V][W];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t c = (int64_t)g * a.width + (v * T + t) * W;
    const bool in = lane_in && v * T + t < nvec;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      w[v][j] = 1.0f;
      b[v][j] = dw[v][j] = db[v][j] = 0.0f;
    }
    if (in && a.w) load_w<float, W>(a.w, c, w[v]);
    if (in && a.b) load_w<float, W>(a.b, c, b[v]);
  }
  const float inv = 1.0f / (float)a.width;
  int turn = 0;
  // (whole waves run the same trips, workgroups where a group takes one)
  for (int64_t r0 = (rb * kWaves + (T > 64 ? 0 : threadIdx.x / 64)) * rw; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + (T > 64 ? 0 : sub / gw);
    const bool some = lane_in && row < a.rows;
    const int64_t base = (row * a.G + g) * a.width;
    float x[V][W], z[V][W], d[V][W];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * T + t) * W;
      const bool in = some && v * T + t < nvec;
#pragma unroll
      for (int j = 0; j < W; ++j) x[v][j] = z[v][j] = d[v][j] = 0.0f;
      if (in) {
        load_w<IoT, W>(a.x, base + c, x[v]);
        load_w<IoT, W>(a.dy, base + c, d[v]);
        if (a.z) load_w<IoT, W>(a.z, row * a.z_stride + (int64_t)g * a.width + c, z[v]);
      }
    }
    // two sets of LDS words in turn: a fast wave's next row does not overwrite what a slow one reads
    const float rstd = normalise<W, T, V>(a, x, t, red[turn]);
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(some && v * T + t < nvec)) continue;
      if (a.z) {
        float dz[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float n = fmaf(x[v][j], w[v][j], b[v][j]), s = sigmoid(z[v][j]);
          dz[j] = d[v][j] * n * s * fmaf(z[v][j], 1.0f - s, 1.0f);
          d[v][j] *= z[v][j] * s;
        }
        store_w<IoT, W>(a.dz, base + (v * T + t) * W, dz);
      } else if (a.silu) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float n = fmaf(x[v][j], w[v][j], b[v][j]), s = sigmoid(n);
          d[v][j] *= s * fmaf(n, 1.0f - s, 1.0f);
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        dw[v][j] = fmaf(d[v][j], x[v][j], dw[v][j]);
        db[v][j] += d[v][j];
        d[v][j] *= w[v][j];
        sg += d[v][j];
        sgx = fmaf(d[v][j], x[v][j], sgx);
      }
    }
    sg = a.center ? group_reduce<T>(sg, red[turn][kReds]) * inv : 0.0f;
    sgx = group_reduce<T>(sgx, red[turn][kReds + 1]) * inv;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(some && v * T + t < nvec)) continue;
#pragma unroll
      for (int j = 0; j < W; ++j) d[v][j] = rstd * (d[v][j] - sg - x[v][j] * sgx);
      store_w<IoT, W>(a.y, base + (v * T + t) * W, d[v]);
    }
  }
  if (!a.want_w && !a.want_b) return;
  const int64_t dim = (int64_t)a.G * a.width;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? a.want_b : a.want_w)) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[W];
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = k ? db[v][j] : dw[v][j];
      if constexpr (T <= 64) {   // the waves' sums, and of the rows that a wave takes at a time, in a fixed order
        __syncthreads();
#pragma unroll
        for (int j = 0; j < W; ++j) sums[threadIdx.x][j] = f[j];
        __syncthreads();
        if (threadIdx.x >= 64 || sub / gw != 0) continue;
        for (int i = 1; i < kWaves * rw; ++i) {
          const int at = (i / rw) * 64 + (i % rw) * gw * T + threadIdx.x;
#pragma unroll
          for (int j = 0; j < W; ++j) f[j] += sums[at][j];
        }
      }
      if (lane_in && v * T + t < nvec)
        store_w<float, W>(a.part, (rb * 2 + k) * dim + (int64_t)g * a.width + (v * T + t) * W, f);
    }
  }
}

// dweight and dbias: sums of part[0 .. n)[k][c], 16 columns a workgroup, 64 threads a column
__global__ __launch_bounds__(1024) void group_norm_sums_kernel(const float* part, float* dw, float* db, int n, int64_t dim) {
  __shared__ float red[64][17];
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int col = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + col;
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (int k = g; k < n; k += 64) s += part[(2 * (int64_t)k + blockIdx.y) * dim + c];
  }
  red[g][col] = s;
  __syncthreads();
  for (int h = 32; h; h >>= 1) {
    if (g < h) red[g][col] += red[g + h][col];
    __syncthreads();
  }
  if (g == 0 && c < dim) out[c] = red[0][col];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The shapes a group is run in: as many lanes as hold it in one access each, a workgroup past 1024 channels;
// groups off 16-byte alignment element by element.
enum { kV8, kV16, kV32, kV64, kV64x2, kG1, kG2, kG4, kOdd8, kOdd64, kOddG, kOddG4 };

int group_shape(int width, bool vec) {
  if (vec) return width <= 64 ? kV8 : width <= 128 ? kV16 : width <= 256 ? kV32 : width <= 512 ? kV64 : width <= 1024 ? kV64x2
                : width <= 2048 ? kG1 : width <= 4096 ? kG2 : kG4;
  return width <= 32 ? kOdd8 : width <= 512 ? kOdd64 : width <= 2048 ? kOddG : kOddG4;
}

int lanes_of(int shape) {
  const int n[] = {8, 16, 32, 64, 64, 256, 256, 256, 8, 64, 256, 1024};
  return n[shape];
}

#define MSCAN_GROUP_SHAPE(SHAPE, KERNEL, W, T, V, ...)                                                     \
  case SHAPE:                                                                                              \
    hipLaunchKernelGGL((KERNEL<IoT, W, T, V>), grid, dim3(threads_of(T)), 0, s, __VA_ARGS__);              \
    break;
#define MSCAN_GROUP_SHAPES(KERNEL, ...)                        \
  switch (shape) {                                             \
    MSCAN_GROUP_SHAPE(kV8, KERNEL, 8, 8, 1, __VA_ARGS__)       \
    MSCAN_GROUP_SHAPE(kV16, KERNEL, 8, 16, 1, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kV32, KERNEL, 8, 32, 1, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kV64, KERNEL, 8, 64, 1, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kV64x2, KERNEL, 8, 64, 2, __VA_ARGS__)   \
    MSCAN_GROUP_SHAPE(kG1, KERNEL, 8, 256, 1, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kG2, KERNEL, 8, 256, 2, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kG4, KERNEL, 8, 256, 4, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kOdd8, KERNEL, 1, 8, 4, __VA_ARGS__)     \
    MSCAN_GROUP_SHAPE(kOdd64, KERNEL, 1, 64, 8, __VA_ARGS__)   \
    MSCAN_GROUP_SHAPE(kOddG, KERNEL, 1, 256, 8, __VA_ARGS__)   \
    MSCAN_GROUP_SHAPE(kOddG4, KERNEL, 1, 1024, 8, __VA_ARGS__) \
    default: return hipErrorInvalidValue;                      \
  }

GArgs args_of(const GroupNormArgs& p) {
  GArgs a{};
  a.dy = p.dy; a.x = p.x; a.z = p.z; a.w = p.weight; a.b = p.bias; a.y = p.y; a.dz = p.dz;
  a.part = static_cast<float*>(p.workspace); a.rows = p.rows; a.z_stride = p.z_stride; a.G = (int)p.groups;
  a.width = (int)p.width; a.center = p.center; a.silu = p.silu; a.want_w = p.dweight != nullptr;
  a.want_b = p.dbias != nullptr; a.eps = p.eps;
  return a;
}

bool by_eights(const GroupNormArgs& p) {
  return p.width % 8 == 0 && (!p.z || p.z_stride % 8 == 0) && aligned16(p.dy) && aligned16(p.x) && aligned16(p.z) &&
         aligned16(p.weight) && aligned16(p.bias) && aligned16(p.y) && aligned16(p.dz);
}

template <typename IoT>
hipError_t run_fwd(const GroupNormArgs& p, hipStream_t s) {
  const GArgs a = args_of(p);
  const int shape = group_shape(a.width, by_eights(p));
  const int per = std::max(1, 256 / lanes_of(shape));
  const dim3 grid((unsigned)((a.rows * a.G + per - 1) / per));
  MSCAN_GROUP_SHAPES(group_norm_fwd_kernel, a)
  return hipGetLastError();
}

template <typename IoT>
hipError_t run_bwd(const GroupNormArgs& p, hipStream_t s) {
  const GArgs a = args_of(p);
  int64_t parts = 0;
  if (a.rows > 0) {
    const int shape = group_shape(a.width, by_eights(p)), lanes = lanes_of(shape);
    const int gw = lanes > 64 ? 1 : std::min(a.G, 64 / lanes), rows_at = lanes > 64 ? 1 : 4 * (64 / lanes / gw);
    const int cblocks = (a.G + gw - 1) / gw;
    parts = std::min((a.rows + rows_at - 1) / rows_at, group_norm_bwd_parts(a.rows, a.G, a.width));
    const dim3 grid((unsigned)(parts * cblocks));
    MSCAN_GROUP_SHAPES(group_norm_bwd_kernel, a, gw, cblocks)
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.dweight && !p.dbias) return hipSuccess;
  const int64_t dim = (int64_t)a.G * a.width;
  hipLaunchKernelGGL(group_norm_sums_kernel, dim3((unsigned)((dim + 15) / 16), 2), dim3(1024), 0, s, a.part, p.dweight,
                     p.dbias, (int)parts, dim);
  return hipGetLastError();
}

}  // namespace

// 2048 workgroups or so: each takes some 512 columns (8 lanes of 8 elements to a workgroup's 2048)
int64_t group_norm_bwd_parts(int64_t rows, int64_t groups, int64_t width) {
  const int64_t dim = groups * width;
  return std::max<int64_t>(1, std::min<int64_t>(rows, 2048 / std::max<int64_t>(1, dim / 512)));
}

hipError_t launch_group_norm_fwd(const GroupNormArgs& a, hipStream_t stream) {
  return a.io_bf16 ? run_fwd<uint16_t>(a, stream) : run_fwd<float>(a, stream);
}

hipError_t launch_group_norm_bwd(const GroupNormArgs& a, hipStream_t stream) {
  return a.io_bf16 ? run_bwd<uint16_t>(a, stream) : run_bwd<float>(a, stream);
}

}  // namespace mscan
