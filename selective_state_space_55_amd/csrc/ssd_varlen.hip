// ssd_varlen.hip -- multi-head SSM with a scalar decay per head over packed
// sequences (prompts), with a state per request slot, on gfx950 matrix cores.
//
// Per sequence, head h (group g of B and C), with a_t = exp(Delta_t A_h) and the
// input weight w_t ((a_t - 1) / A_h, or Delta_t for the Euler input term):
//
//   S_t = a_t S_{t-1} + w_t B_t x_t^T          (N x P)
//   y_t = (S_t^T C_t + D_h x_t) SiLU(z_t)
//
// in chunks of Q = 64 tokens (State space models and Mamba, jonathanding.github.io,
// §5): with cum_i the running sum of log a in the chunk,
//
//   Y^T = S_in^T C^T diag(e^cum) + X^T M^T,  M_ij = (C B^T)_ij e^(cum_i - cum_j) w_j (j <= i)
//   S_out = e^cum_Q S_in + B^T (diag(e^(cum_Q - cum_j) w_j) X)
//
// Mapping.  A workgroup of 4 waves owns one (piece of a sequence, head, slice of P
// = 64 or 32 channels) and walks its chunks.  Every product is a 32x32x16 MFMA on
// bf16 operands with fp32 accumulation; wave w has output rows p-tile pb = w mod PB
// and tokens i-tile ib = w / PB, and a part of S (p-tile pb, some of the n-tiles) in
// its accumulators.  What stays in registers:
//   C      as the B operand of both C B^T and S^T C^T: a lane's 16-byte pieces of one
//          token's row, loaded straight from memory
//   M      C B^T comes out as (B C^T)[j][i], lane = column i, rows j in runs of four; the
//          order of an MFMA's k index is free as long as both operands agree, so the
//          masked, decayed tile is the B operand of X^T M^T as it is, and X^T (and B^T and
//          X in the state update) are read from LDS in that order of tokens
//   Y      leaves as Y^T: a lane holds four consecutive channels of its token, two lanes
//          trade halves (v_permlane32_swap), and 16 bytes go out per lane
// In LDS: the chunk's B and x as loaded, S^T as bf16 hi + lo for the readout (~2^-17), and
// the decay terms, 65 KB at (N, P) = (128, 64), so that two workgroups share a CU and one's
// waits overlap the other's work.  The scaled x of the state update is split into three
// bf16 parts by truncation (8 bits each: exact), so the state keeps fp32's accuracy over a
// long prompt; e^(cum_Q - cum_j) is taken from the sum of the logs behind j, not from a
// difference of two long sums.
#include "internal.h"
#include "io.h"
#include "mfma.h"
#include "packed.h"

#include <algorithm>

namespace mscan {
namespace {

constexpr int kQ = 64;   // tokens per chunk

struct VArgs {
  Packed seq;
  const uint16_t* x;
  const uint16_t* dt;
  const float* A_log;
  const uint16_t* B;
  const uint16_t* C;
  const float* D;
  const uint16_t* z;
  const float* dt_bias;
  float* state;
  uint16_t* y;
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;
  int64_t piece;      // tokens per piece, 0: whole sequences
  float* ws_state;    // (pieces, H, P, N): a piece's own state, then the state that enters it
  float* ws_decay;    // (pieces, H): sum of log a over a piece
  int H, HP, G, S;    // heads, head dim, groups, P-channel slices per head
  int softplus, euler;
};

template <int N, int P>
struct Lds {
  static constexpr int kRowB = N + 16;                 // pitches that put the transposing reads' rows
  static constexpr int kRowX = P == 64 ? 96 : 40;      // in different banks
  static constexpr int kRowS = N + 8;
  static constexpr int kHalves = kQ * kRowB + kQ * kRowX + 2 * P * kRowS;
  static constexpr int kTerms = 4 * kQ;                // cum | e^cum | e^(cum_Q - cum) w | w
  static constexpr size_t bytes() { return 2 * (size_t)kHalves + 4 * (size_t)(2 * kTerms + 4); }
};

// k slice s of 16 tokens in the order an accumulator holds its rows: lane half h gets tokens
// 16 s + 4 h .. + 3, then 16 s + 8 + 4 h .. + 3, of column n0 + l % 32
__device__ __forceinline__ bf16x8 opnd_acc_order(const uint16_t* base, int stride, int s, int n0, int lane) {
  const int g = lane >> 4, m = lane & 15;
  const uint16_t* p = base + (16 * s + 4 * (g >> 1) + (m >> 2)) * stride + n0 + 16 * (g & 1) + 4 * (m & 3);
  const uint2 lo = lds_tr16(p);
  const uint2 hi = lds_tr16(p + 8 * stride);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

// the upper halves of two words
__device__ __forceinline__ uint32_t hi16x2(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float trunc16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int N, int P>
__global__ __launch_bounds__(256, 2) void ssd_varlen_kernel(VArgs a) {
  using L = Lds<N, P>;
  constexpr int PB = P / 32;                            // p-tiles
  constexpr int TPW = (N / 32) * PB >= 4 ? (N / 32) * PB / 4 : 1;   // S tiles per wave
  constexpr int NS = N / 16;                            // k slices over the states
  extern __shared__ __align__(16) uint16_t sm[];
  uint16_t* Bs = sm;
  uint16_t* Xs = Bs + kQ * L::kRowB;
  uint16_t* Sh = Xs + kQ * L::kRowX;
  uint16_t* Sl = Sh + P * L::kRowS;
  float* terms = reinterpret_cast<float*>(Sl + P * L::kRowS);   // two sets
  float* atots = terms + 2 * L::kTerms;                         // e^cum_Q of the two sets
  lds_poison(sm, (int)L::bytes());

  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h32 = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int HS = a.H * a.S;
  const int hs = blockIdx.x % HS;
  const int64_t item = blockIdx.x / HS;
  const int h = hs / a.S, pslice = (hs % a.S) * P, g = h / (a.H / a.G);

  // the sequence and its tokens of this workgroup
  const int64_t s = uniform64(item);
  const int64_t t_first = seq_offset(a.seq, s), t_end = seq_offset(a.seq, s + 1);
  if (t_first >= t_end) return;   // a sequence without tokens leaves its slot as it is
  const int64_t slot = seq_slot(a.seq, s);
  float* const slot_state = slot < 0 ? nullptr : a.state + ((slot * a.H + h) * a.HP + pslice) * N;
  const bool started = slot >= 0 && seq_position(a.seq, s) > 0;
  const int64_t nchunk = (t_end - t_first + kQ - 1) / kQ;

  const float Ah = -expf(a.A_log[h]);
  const float Dh = a.D ? a.D[h] : 0.0f;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const uint16_t* xg = a.x + (int64_t)h * a.HP + pslice;
  const uint16_t* zg = a.z ? a.z + (int64_t)h * a.HP + pslice : nullptr;
  uint16_t* yg = a.y + (int64_t)h * a.HP + pslice;
  const int64_t y_stride = (int64_t)a.H * a.HP;
  const uint16_t* Bg = a.B + (int64_t)g * N;
  const uint16_t* Cg = a.C + (int64_t)g * N;

  // Tokens t0 .. t0 + 63 of an array with `stride` elements per token, `width` of which are this
  // workgroup's: a buffer that ends with the last of them inside the sequence, so that loads past
  // it give 0 and stores past it are dropped.
  auto rows = [&](const uint16_t* base, int64_t t0, int64_t stride, int width) {
    const int64_t left = t_end - t0, n = left < kQ ? left : kQ;
    const int64_t bytes = left <= 0 ? 0 : ((n - 1) * stride + width) * 2;
    return make_rsrc(base + (left <= 0 ? 0 : t0 * stride), (int)bytes);
  };
  auto ld16 = [&](__amdgpu_buffer_rsrc_t r, int off) -> uint4 {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  };

  // staging pieces: B rows of N / 8 16-byte pieces, x rows of P / 8
  constexpr int kBr = kQ * (N / 8) / 256, kXr = kQ * (P / 8) / 256;
  static_assert(kBr >= 1 && kXr >= 1, "a piece per thread at least");
  uint4 bq[kBr], xq[kXr];
  uint32_t dtq = 0;
  auto load_tiles = [&](int64_t t0) {
    const auto rb = rows(Bg, t0, a.b_stride, N), rx = rows(xg, t0, a.x_stride, P);
#pragma unroll
    for (int r = 0; r < kBr; ++r) {
      const int e = tid + 256 * r;
      bq[r] = ld16(rb, ((e / (N / 8)) * (int)a.b_stride + (e % (N / 8)) * 8) * 2);
    }
#pragma unroll
    for (int r = 0; r < kXr; ++r) {
      const int e = tid + 256 * r;
      xq[r] = ld16(rx, ((e / (P / 8)) * (int)a.x_stride + (e % (P / 8)) * 8) * 2);
    }
  };
  auto store_tiles = [&]() {
#pragma unroll
    for (int r = 0; r < kBr; ++r) {
      const int e = tid + 256 * r;
      *reinterpret_cast<uint4*>(Bs + (e / (N / 8)) * L::kRowB + (e % (N / 8)) * 8) = bq[r];
    }
#pragma unroll
    for (int r = 0; r < kXr; ++r) {
      const int e = tid + 256 * r;
      *reinterpret_cast<uint4*>(Xs + (e / (P / 8)) * L::kRowX + (e % (P / 8)) * 8) = xq[r];
    }
  };
  constexpr int kDtWave = 3;
  auto load_dt = [&](int64_t t0) {
    if (w == kDtWave) dtq = __builtin_amdgcn_raw_buffer_load_b16(rows(a.dt + h, t0, a.dt_stride, 1), lane * (int)a.dt_stride * 2, 0, 0);
  };
  // one wave turns a chunk's dt into its decay terms; past the end a = 1 and w = 0
  auto dt_terms = [&](int64_t t0, int set) {
    if (w != kDtWave) return;
    const float v = bf(dtq) + bias;
    float delta = a.softplus ? softplus_log2e(v) * 0.6931471805599453f : v;
    delta = t0 + lane < t_end ? delta : 0.0f;
    const float la = delta * Ah;
    const float wj = a.euler ? delta : Ah != 0.0f ? expm1f(la) / Ah : delta;
    const float cum = wave_prefix_sum(la);
    const float rev = wave_prefix_sum(__shfl(la, 63 - lane));   // from the chunk's end
    const float from = __shfl(rev, 63 - lane);                  // token lane .. the last
    const float next = __shfl_down(from, 1);                    // every lane takes part
    const float behind = lane == 63 ? 0.0f : next;              // lane + 1 .. the last
    float* o = terms + set * L::kTerms;
    o[lane] = cum;
    o[kQ + lane] = expf(cum);
    o[2 * kQ + lane] = expf(behind) * wj;
    o[3 * kQ + lane] = wj;
    if (lane == 63) atots[set] = expf(cum);
  };

  // ---- roles: p-tile pb; the wave's tokens ib of Y, and its n-tiles of S ----
  const int pb = w % PB, ib = w / PB;
  const bool has_y = ib < 2;
  const bool has_s = (w / PB) * TPW < N / 32;
  const int nb = (w / PB) * TPW;
  const int i_tok = (ib & 1) * 32 + l32;   // this lane's token of Y^T

  f32x16 S[TPW];
#pragma unroll
  for (int k = 0; k < TPW; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (has_s && started)
        v = *reinterpret_cast<const float4*>(slot_state + (int64_t)(pb * 32 + l32) * N + (nb + k) * 32 + 8 * q + 4 * h32);
      S[k][4 * q] = v.x; S[k][4 * q + 1] = v.y; S[k][4 * q + 2] = v.z; S[k][4 * q + 3] = v.w;
    }
  // S^T to LDS as hi (truncated) and lo (the rest, rounded)
  auto write_S = [&]() {
    if (!has_s) return;
#pragma unroll
    for (int k = 0; k < TPW; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v0 = S[k][4 * q], v1 = S[k][4 * q + 1], v2 = S[k][4 * q + 2], v3 = S[k][4 * q + 3];
        const int o = (pb * 32 + l32) * L::kRowS + (nb + k) * 32 + 8 * q + 4 * h32;
        *reinterpret_cast<uint2*>(Sh + o) = make_uint2(hi16x2(v0, v1), hi16x2(v2, v3));
        *reinterpret_cast<uint2*>(Sl + o) =
            make_uint2(pack_bf16x2(v0 - trunc16(v0), v1 - trunc16(v1)), pack_bf16x2(v2 - trunc16(v2), v3 - trunc16(v3)));
      }
  };

  // C of the wave's tokens: slice s is states 16 s + 8 h .. + 7
  bf16x8 cf[NS];
  auto load_c = [&](int64_t t0) {
    if (!has_y) return;
    const auto rc = rows(Cg, t0, a.c_stride, N);
    const int off = (i_tok * (int)a.c_stride + 8 * h32) * 2;
#pragma unroll
    for (int k = 0; k < NS; ++k) cf[k] = __builtin_bit_cast(bf16x8, ld16(rc, off + 32 * k));
  };

  load_tiles(t_first);
  load_dt(t_first);
  load_c(t_first);
  dt_terms(t_first, 0);
  load_dt(t_first + kQ);

  for (int64_t c = 0; c < nchunk; ++c) {
    const int64_t t0 = t_first + c * kQ;
    const int set = (int)(c & 1);
    const float* cum = terms + set * L::kTerms;
    const float* ecum = cum + kQ;
    const float* scl = ecum + kQ;
    const float* wv = scl + kQ;
    store_tiles();
    write_S();
    lds_barrier();
    // the next chunk's tiles, and this one's gate
    load_tiles(t0 + kQ);
    uint4 zq[2] = {};
    const int yo = (i_tok * (int)y_stride + pb * 32 + 8 * h32) * 2;
    if (has_y && zg) {
      const auto rz = rows(zg, t0, a.z_stride, P);
      const int zo = (i_tok * (int)a.z_stride + pb * 32 + 8 * h32) * 2;
      zq[0] = ld16(rz, zo);
      zq[1] = ld16(rz, zo + 32);
    }
    dt_terms(t0 + kQ, set ^ 1);
    load_dt(t0 + 2 * kQ);

    bf16x8 xf[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) xf[k] = opnd_acc_order(Xs, L::kRowX, k, pb * 32, lane);
    if (has_y) {
      // S_in^T C^T, columns scaled by e^cum
      f32x16 y = {};
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const int o = (pb * 32 + l32) * L::kRowS + 16 * k + 8 * h32;
        y = mfma(lds_b8(Sl + o), cf[k], y);
        y = mfma(lds_b8(Sh + o), cf[k], y);
      }
      const float ei = ecum[i_tok], ci = cum[i_tok];
#pragma unroll
      for (int r = 0; r < 16; ++r) y[r] *= ei;
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        if (jb > ib) break;
        f32x16 m = {};
#pragma unroll
        for (int k = 0; k < NS; ++k) m = mfma(lds_b8(Bs + (jb * 32 + l32) * L::kRowB + 16 * k + 8 * h32), cf[k], m);
        uint32_t mw[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j0 = jb * 32 + 8 * q + 4 * h32;
          const float4 cj = *reinterpret_cast<const float4*>(cum + j0);
          const float4 wj = *reinterpret_cast<const float4*>(wv + j0);
          const float cja[4] = {cj.x, cj.y, cj.z, cj.w}, wja[4] = {wj.x, wj.y, wj.z, wj.w};
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // exp(-200) is 0 in fp32: the tokens behind i
            const float d = jb < ib || j0 + r <= i_tok ? ci - cja[r] : -200.0f;
            v[r] = m[4 * q + r] * __expf(d) * wja[r];
          }
          mw[2 * q] = pack_bf16x2(v[0], v[1]);
          mw[2 * q + 1] = pack_bf16x2(v[2], v[3]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          y = mfma(xf[2 * jb + k], __builtin_bit_cast(bf16x8, make_uint4(mw[4 * k], mw[4 * k + 1], mw[4 * k + 2], mw[4 * k + 3])), y);
      }
      // + D x, gate, and out: channels 8 q + 4 h .. + 3 of the lane's token
      uint32_t zw[8];
      const uint32_t zr[8] = {zq[0].x, zq[0].y, zq[0].z, zq[0].w, zq[1].x, zq[1].y, zq[1].z, zq[1].w};
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t lo = zr[4 * k + j], up = zr[4 * k + 2 + j];
          swap32(lo, up);
          zw[4 * k + j] = lo;
          zw[4 * k + 2 + j] = up;
        }
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 xv = *reinterpret_cast<const uint2*>(Xs + i_tok * L::kRowX + pb * 32 + 8 * q + 4 * h32);
        const uint32_t xw[2] = {xv.x, xv.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v0 = fmaf(Dh, bf16_lo(xw[j]), y[4 * q + 2 * j]), v1 = fmaf(Dh, bf16_hi(xw[j]), y[4 * q + 2 * j + 1]);
          if (zg) {
            v0 *= silu(bf16_lo(zw[2 * q + j]));
            v1 *= silu(bf16_hi(zw[2 * q + j]));
          }
          o[2 * q + j] = pack_bf16x2(v0, v1);
        }
      }
      const auto ry = rows(yg, t0, y_stride, P);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        swap32(o[4 * k], o[4 * k + 2]);
        swap32(o[4 * k + 1], o[4 * k + 3]);
        typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]}, ry, yo + 32 * k, 0, 0);
      }
    }
    load_c(t0 + kQ);
    if (has_s) {
      const float at = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(atots[set])));
#pragma unroll
      for (int k = 0; k < TPW; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[k][r] *= at;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 s0 = *reinterpret_cast<const float4*>(scl + 16 * k + 4 * h32);
        const float4 s1 = *reinterpret_cast<const float4*>(scl + 16 * k + 8 + 4 * h32);
        const uint4 xv = __builtin_bit_cast(uint4, xf[k]);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
        const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v0 = bf16_lo(xw[j]) * sc[2 * j], v1 = bf16_hi(xw[j]) * sc[2 * j + 1];
          const float r0 = v0 - trunc16(v0), r1 = v1 - trunc16(v1);
          hi[j] = hi16x2(v0, v1);
          mid[j] = hi16x2(r0, r1);
          lo[j] = hi16x2(r0 - trunc16(r0), r1 - trunc16(r1));
        }
        const bf16x8 xh = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        const bf16x8 xm = __builtin_bit_cast(bf16x8, make_uint4(mid[0], mid[1], mid[2], mid[3]));
        const bf16x8 xl = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
        for (int n = 0; n < TPW; ++n) {
          const bf16x8 bt = opnd_acc_order(Bs, L::kRowB, k, (nb + n) * 32, lane);
          S[n] = mfma(bt, xl, S[n]);
          S[n] = mfma(bt, xm, S[n]);
          S[n] = mfma(bt, xh, S[n]);
        }
      }
    }
    lds_barrier();   // the tiles, S and the terms of this chunk have been read
  }

  if (slot_state && has_s) {
#pragma unroll
    for (int k = 0; k < TPW; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(slot_state + (int64_t)(pb * 32 + l32) * N + (nb + k) * 32 + 8 * q + 4 * h32) =
            make_float4(S[k][4 * q], S[k][4 * q + 1], S[k][4 * q + 2], S[k][4 * q + 3]);
  }
}

template <int N, int P>
hipError_t run(VArgs a, const SsdVarlenPlan& p, hipStream_t s) {
  a.S = a.HP / P;
  const size_t lds = Lds<N, P>::bytes();
  hipError_t e = hipFuncSetAttribute((const void*)ssd_varlen_kernel<N, P>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((ssd_varlen_kernel<N, P>), dim3((unsigned)(p.pieces * a.H * a.S)), dim3(256), lds, s, a);
  return hipGetLastError();
}

}  // namespace

SsdVarlenPlan make_ssd_varlen_plan(int64_t nseq, int64_t total, int64_t nheads, int64_t headdim, int64_t dstate) {
  SsdVarlenPlan p{};
  p.pieces = nseq;
  return p;
}

hipError_t launch_ssd_varlen(const SsdVarlenArgs& p, const SsdVarlenPlan& plan, hipStream_t stream) {
  VArgs a{};
  a.seq.cu = p.cu; a.seq.slots = p.slots; a.seq.positions = p.positions;
  a.seq.nseq = p.nseq; a.seq.total = p.total; a.seq.nslots = p.nslots;
  a.x = static_cast<const uint16_t*>(p.x); a.dt = static_cast<const uint16_t*>(p.dt); a.A_log = p.A_log;
  a.B = static_cast<const uint16_t*>(p.B); a.C = static_cast<const uint16_t*>(p.C); a.D = p.D;
  a.z = static_cast<const uint16_t*>(p.z); a.dt_bias = p.dt_bias; a.state = p.state; a.y = static_cast<uint16_t*>(p.y);
  a.x_stride = p.x_stride; a.dt_stride = p.dt_stride; a.b_stride = p.b_stride; a.c_stride = p.c_stride; a.z_stride = p.z_stride;
  a.H = (int)p.nheads; a.HP = (int)p.headdim; a.G = (int)p.ngroups; a.softplus = p.softplus; a.euler = p.euler;
  const bool p32 = p.headdim % 64 != 0;
  if (p.dstate == 128) return p32 ? run<128, 32>(a, plan, stream) : run<128, 64>(a, plan, stream);
  return p32 ? run<64, 32>(a, plan, stream) : run<64, 64>(a, plan, stream);
}

}  // namespace mscan
