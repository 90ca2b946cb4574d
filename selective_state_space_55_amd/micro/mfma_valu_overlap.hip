// mfma_valu_overlap.hip -- whether matrix and vector instructions of two waves overlap on a gfx950 SIMD.
// One workgroup of 8 waves, two per SIMD (waves w and w + 4).  A pass of a loop is two 32x32x16 bf16 MFMAs, or 16
// v_mul_f32 on 8 registers, or both in turn; register operands only.  Reported: s_memtime ticks per pass, per wave.
// Build: hipcc --offload-arch=gfx950 -O3 -Xclang -target-feature -Xclang -packed-fp32-ops -o overlap mfma_valu_overlap.hip
// Buffers: out has one float per thread (512), ticks one long per wave (8).
#include <hip/hip_runtime.h>
#include <cstdio>
#include <cstdlib>
#define CHK(x) do { hipError_t e_ = (x); if (e_ != hipSuccess) { printf("HIP error %s at %d\n", hipGetErrorString(e_), __LINE__); exit(1);} } while (0)
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kPasses = 4096;

enum Work { kNone, kMfma, kValu, kInTurn };

template <bool kM, bool kV>
__device__ __forceinline__ void passes(f32x16& c0, f32x16& c1, float (&v)[8]) {
  bf16x8 a = {}, b = {};
  for (int n = 0; n < kPasses; ++n) {
    if constexpr (kM) c0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c0, 0, 0, 0);
    if constexpr (kV) {
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("v_mul_f32 %0, %0, %0" : "+v"(v[j]));
    }
    if constexpr (kM) c1 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c1, 0, 0, 0);
    if constexpr (kV) {
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("v_mul_f32 %0, %0, %0" : "+v"(v[j]));
    }
  }
}

__global__ __launch_bounds__(512) void run(float* out, long* ticks, int first, int second) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), work = w < 4 ? first : second;
  f32x16 c0 = {}, c1 = {};
  float v[8];
  for (int i = 0; i < 8; ++i) v[i] = threadIdx.x + i;
  __syncthreads();
  const long t0 = __builtin_amdgcn_s_memtime();
  if (work == kMfma) passes<true, false>(c0, c1, v);
  if (work == kValu) passes<false, true>(c0, c1, v);
  if (work == kInTurn) passes<true, true>(c0, c1, v);
  const long t1 = __builtin_amdgcn_s_memtime();
  float s = 0;
  for (int i = 0; i < 16; ++i) s += c0[i] + c1[i];
  for (int i = 0; i < 8; ++i) s += v[i];
  out[threadIdx.x] = s;
  if ((threadIdx.x & 63) == 0) ticks[w] = t1 - t0;
}

int main() {
  float* out;
  long *ticks, h[8];
  CHK(hipMalloc(&out, 512 * sizeof(float)));
  CHK(hipMalloc(&ticks, 8 * sizeof(long)));
  const struct { const char* name; int first, second; } rows[] = {
      {"MFMA | idle", kMfma, kNone}, {"VALU | idle", kValu, kNone}, {"MFMA | MFMA", kMfma, kMfma},
      {"VALU | VALU", kValu, kValu}, {"MFMA | VALU", kMfma, kValu}, {"in turn | idle", kInTurn, kNone},
      {"in turn | in turn", kInTurn, kInTurn}};
  for (const auto& r : rows)
    for (int k = 0; k < 2; ++k) {   // the second launch is reported
      hipLaunchKernelGGL(run, dim3(1), dim3(512), 0, 0, out, ticks, r.first, r.second);
      CHK(hipGetLastError());
      CHK(hipMemcpy(h, ticks, sizeof(h), hipMemcpyDeviceToHost));
      if (k) printf("%-18s ticks per pass: wave 0 %6.1f, wave 4 %6.1f\n", r.name, (double)h[0] / kPasses, (double)h[4] / kPasses);
    }
  CHK(hipFree(out));
  CHK(hipFree(ticks));
  return 0;
}
