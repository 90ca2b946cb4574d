// mfma.h -- device-side helpers of the matrix-core kernels: 32x32x16 bf16
// products, the LDS reads that feed them, and a wave prefix sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ bf16x8 lds_b8(const uint16_t* p) {
  return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float bf(uint32_t h16) { return __uint_as_float(h16 << 16); }

// v from another lane (DPP move; lanes with no source get 0)
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add_src(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}

// inclusive prefix sum over the 64 lanes: shifts by 1, 2, 4, 8 inside each
// 16-lane row, then row 0's total into row 1, rows 0-1's into rows 2-3, etc.
__device__ __forceinline__ float wave_prefix_sum(float v) {
  v += dpp_add_src<0x111, 0xf>(v);   // row_shr:1
  v += dpp_add_src<0x112, 0xf>(v);   // row_shr:2
  v += dpp_add_src<0x114, 0xf>(v);   // row_shr:4
  v += dpp_add_src<0x118, 0xf>(v);   // row_shr:8
  v += dpp_add_src<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
  v += dpp_add_src<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
  return v;
}

typedef short v4i16 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint2 lds_tr16(const uint16_t* p) {
  const v4i16 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(p));
  return __builtin_bit_cast(uint2, r);
}

// Operand of a 32x32x16 MFMA whose k index runs along the rows of a row-major
// bf16 tile: lane l gets rows k0 + 8 (l / 32) .. + 7 of column n0 + l % 32.
// Two transposing reads of 4 rows each; in 16-lane group g the lane
// m = a + 4 kk addresses row k0 + 8 (g / 2) + kk, columns n0 + 16 (g % 2) + 4 a .. + 3.
__device__ __forceinline__ bf16x8 lds_opnd_tr(const uint16_t* base, int stride, int k0, int n0, int lane) {
  const int g = lane >> 4, m = lane & 15;
  const uint16_t* p = base + (k0 + 8 * (g >> 1) + (m >> 2)) * stride + n0 + 16 * (g & 1) + 4 * (m & 3);
  const uint2 lo = lds_tr16(p);
  const uint2 hi = lds_tr16(p + 4 * stride);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

}  // namespace mscan
