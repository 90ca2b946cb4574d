// linear_attention.hip -- linear attention with a fixed decay per head over
// packed or equal sequences, its states and its gradient, on gfx950 matrix cores.
//
// Per sequence and head, lam = exp(log_decay), in chunks of 64 tokens:
//
//   S_t = lam S_{t-1} + k_t v_t^T       (A x B, fp32)
//   o_t = c S_t^T q_t
//
//   O^T  = c (S_in^T Q^T diag(lam^(i+1)) + V^T P^T),  P_ij = (q_i . k_j) lam^(i-j) for j <= i
//   S_out = lam^n S_in + K^T (diag(lam^(n-1-j)) V)
//
// The gradient is the same with the arrays' roles exchanged (R_t: the gradient of S_t, which runs
// from the last token to the first, R_t = lam R_{t+1} + c q_t do_t^T):
//
//   dq_t = c S_t do_t     q, k, v -> do, v, k, the state transposed
//   dk_t = R_t v_t        q, k, v -> v, do, q, last token first
//   dv_t = R_t^T k_t      q, k, v -> k, q, do, last token first
#include "internal.h"
#include "io.h"
#include "mfma.h"
#include "packed.h"

#include <algorithm>

namespace mscan {
namespace {

constexpr int kQ = 64;   // tokens per chunk
constexpr int kOut = 0x7ffffff0;   // a buffer offset past any descriptor's end

struct Role {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* o;
  const float* from;   // (entries, H, V, K): the state that a sequence starts from, or null
  float* to;           // the state it ends with, or null
  float* ws;           // (parts, H, V, K): the states that enter a cut sequence's pieces
  int q_stride, k_stride, v_stride;   // elements between tokens; o has no gaps
  int A, B;            // widths of q and k, and of v and o
  int sa, sb;          // state elements between its rows (A) and columns (B)
  int slabs, slab;     // workgroups that share the columns, and columns of each
  int later;           // last token first
  float c_out, c_in;   // factors of what the state gives to o, and of what goes into it
};

struct LaArgs {
  Packed seq;          // cu null: nseq sequences of len tokens
  const float* log_decay;
  Role role[3];
  int first[3];        // role r's first workgroup of a unit
  int wgs;             // workgroups of a unit
  int nroles;
  int64_t len, units;
  int np;              // equal sequences: pieces of each
  int shift, whole;    // pieces of 2^shift tokens; packed sequences of at most 2^whole are not cut
  int H, KV;
  float scale;
};

__device__ __forceinline__ uint32_t hi16x2(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float trunc16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// index m of 32 with bits 2 and 3 exchanged: where operand row m takes row turn(m) of its array, an accumulator's
// registers 8 s .. 8 s + 7 hold the array's rows 16 s + 8 h .. + 7 (h the lane's half), which is an operand's k order
__device__ __forceinline__ int turn(int m) { return (m & 19) | ((m & 4) << 1) | ((m & 8) >> 1); }

// Operand of a 32x32x16 MFMA whose k index runs along the rows of a row-major tile: lane l gets rows k0 + 8 (l / 32) ..
// + 7 of column n0 + turn(l % 32).  (lds_opnd_tr of mfma.h with the columns' blocks of four exchanged.)
__device__ __forceinline__ bf16x8 opnd_tr(const uint16_t* base, int pitch, int k0, int n0, int lane) {
  const int g = lane >> 4, m = lane & 15, a = m & 3;
  const uint16_t* p = base + (k0 + 8 * (g >> 1) + (m >> 2)) * pitch + n0 + 16 * (g & 1) + 4 * ((a >> 1) | ((a & 1) << 1));
  const uint2 lo = lds_tr16(p);
  const uint2 hi = lds_tr16(p + 4 * pitch);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

__device__ __forceinline__ float power(float l2, float x) { return x == 0.0f ? 1.0f : __builtin_amdgcn_exp2f(x * l2); }

template <int A, int NW, bool kAgg>
struct Lds {
  static constexpr int kRowQ = A + 8, kRowK = A + 16, kRowV = NW * 32 + 16;
  static constexpr int kQs = kAgg ? 0 : kQ * kRowQ, kKs = kQ * kRowK, kVs = kQ * kRowV;
  static constexpr size_t bytes() { return 2 * (size_t)(kQs + kKs + kVs) + 4 * 2 * kQ; }
};

__device__ __forceinline__ int64_t part_of(int64_t b, int64_t s) { return b + min(b, s); }

// A sequence's piece: its tokens, its part of the workspace, and whether it is alone
struct Piece {
  int64_t s, first, end, part;
  int64_t k, n;   // number, and pieces of the sequence
};

// kAgg: only the state that a piece would end with from zero
template <int A, int NW, bool kAgg>
__global__ __launch_bounds__(64 * NW, A == 256 ? 1 : 2) void linear_attention_kernel(LaArgs a) {
  using L = Lds<A, NW, kAgg>;
  constexpr int NT = A / 32, NS = A / 16, kThreads = 64 * NW;
  extern __shared__ __align__(16) uint16_t sm[];
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h32 = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint16_t* Qs = sm;
  uint16_t* Ks = Qs + L::kQs;
  uint16_t* Vs = Ks + L::kKs;
  float* into = reinterpret_cast<float*>(Vs + L::kVs);   // lam^(what follows in the chunk), by token
  float* half = into + kQ;                               // lam^(32 - j) for the first 32 tokens
  lds_poison(sm, (int)L::bytes());

  // eight units at a time, each unit's workgroups on one XCD
  const int64_t group = blockIdx.x / (8 * a.wgs);
  const int in_group = blockIdx.x % (8 * a.wgs);
  const int64_t unit = group * 8 + in_group % 8;
  if (unit >= a.units) return;
  const int wg = in_group / 8;
  int ri = 0;
  if (a.nroles > 1 && wg >= a.first[1]) ri = 1;
  if (a.nroles > 2 && wg >= a.first[2]) ri = 2;
  const Role& R = a.role[ri];
  const int b0 = (wg - a.first[ri]) * R.slab;
  const int h = (int)(unit % a.H);
  const int64_t number = unit / a.H;

  int64_t s, start, stop, k, np;
  if (a.seq.cu) {
    const Run run = kAgg ? find_run<true>(a.seq, number, a.shift) : locate_run<false>(a.seq, number, a.shift);
    if (run.s < 0) return;
    s = run.s; start = run.start; stop = max(run.start, run.stop); k = run.k;
    const bool cut = stop - start > (int64_t)1 << a.whole;
    if (!cut && (kAgg || k > 0)) return;
    np = cut ? (stop - start + ((int64_t)1 << a.shift) - 1) >> a.shift : 1;
    if (k >= np) return;
  } else {
    const int64_t per = kAgg ? a.np - 1 : a.np;
    s = number / per; k = number % per; np = a.np;
    start = s * a.len; stop = start + a.len;
  }
  const bool later = R.later != 0;
  if (kAgg && later) ++k;   // a piece that others precede
  const int64_t t_first = np == 1 ? start : start + (k << a.shift);
  const int64_t t_end = np == 1 ? stop : min(stop, t_first + ((int64_t)1 << a.shift));
  const int64_t part = (a.seq.cu ? part_of(start >> a.shift, s) : s * np) + k;
  const int64_t nchunk = (t_end - t_first + kQ - 1) / kQ;
  const int A_ = R.A, cols = min(R.slab, R.B - b0);
  const bool live = w * 32 < cols;

  const float ld = a.log_decay[h], l2 = ld * 1.4426950408889634f;
  const float e = later ? 0.0f : 1.0f;   // decays between a token's entry and the state that it reads

  const uint16_t* qb = kAgg ? nullptr : R.q + (int64_t)h * A_;
  const uint16_t* kb = R.k + (int64_t)h * A_;
  const uint16_t* vb = R.v + (int64_t)h * R.B + b0;

  auto tokens = [&](int64_t c, int64_t& t0) -> int {   // of chunk c, in the order they are taken
    if (later) {
      const int64_t hi = t_end - c * kQ;
      t0 = max(t_first, hi - kQ);
      return (int)(hi - t0);
    }
    t0 = t_first + c * kQ;
    return (int)min(t_end - t0, (int64_t)kQ);
  };
  auto ld16 = [&](__amdgpu_buffer_rsrc_t r, int off) -> uint4 {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  };

  constexpr int kCpr = A / 8, kRpp = kThreads / kCpr, kR = kQ / kRpp;   // q, k: 16-byte pieces per row, rows per pass
  constexpr int kVpr = NW * 4, kVr = kQ * kVpr / kThreads;              // v: 16 rows per pass
  const int kr = tid / kCpr, kc = (tid % kCpr) * 8;
  const int vr = tid / kVpr, vc = (tid % kVpr) * 8;
  const bool k_in = kc < A_, v_in = vc < cols;
  uint4 qq[kAgg ? 1 : kR], kq[kR], vq[kVr];
  auto load = [&](int64_t c) {
    int64_t t0;
    const int n = tokens(c, t0);
    const auto rk = make_rsrc(kb + t0 * R.k_stride, ((n - 1) * R.k_stride + A_) * 2);
    const auto rv = make_rsrc(vb + t0 * R.v_stride, ((n - 1) * R.v_stride + cols) * 2);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int i = kr + r * kRpp, row = later ? n - 1 - i : i;
      const bool in = k_in && i < n;
      kq[r] = ld16(rk, in ? (row * R.k_stride + kc) * 2 : kOut);
    }
    if constexpr (!kAgg) {
      const auto rq = make_rsrc(qb + t0 * R.q_stride, ((n - 1) * R.q_stride + A_) * 2);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int i = kr + r * kRpp, row = later ? n - 1 - i : i;
        const bool in = k_in && i < n;
        qq[r] = ld16(rq, in ? (row * R.q_stride + kc) * 2 : kOut);
      }
    }
#pragma unroll
    for (int r = 0; r < kVr; ++r) {
      const int i = vr + r * 16, row = later ? n - 1 - i : i;
      const bool in = v_in && i < n;
      vq[r] = ld16(rv, in ? (row * R.v_stride + vc) * 2 : kOut);
    }
  };
  auto store_tiles = [&]() {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      *reinterpret_cast<uint4*>(Ks + (kr + r * kRpp) * L::kRowK + kc) = kq[r];
      if constexpr (!kAgg) *reinterpret_cast<uint4*>(Qs + (kr + r * kRpp) * L::kRowQ + kc) = qq[r];
    }
#pragma unroll
    for (int r = 0; r < kVr; ++r) *reinterpret_cast<uint4*>(Vs + (vr + r * 16) * L::kRowV + vc) = vq[r];
  };

  if (nchunk > 0) load(0);

  // the lane's column of the state, and the entry it comes from
  const int64_t bcol = b0 + w * 32 + turn(l32);
  const bool has_col = live && w * 32 + turn(l32) < cols;
  const int64_t entry = a.seq.slots ? seq_slot(a.seq, s) : s;
  const bool started = entry >= 0 && (!a.seq.positions || a.seq.positions[s] > 0);
  const int64_t at_head = (int64_t)h * a.KV, row_state = (int64_t)a.H * a.KV;
  const float* from = kAgg ? nullptr : np > 1 ? R.ws + part * row_state + at_head
                    : R.from && started ? R.from + entry * row_state + at_head : nullptr;
  f32x16 S[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int64_t ra = n * 32 + g * 16 + h32 * 8;
      const bool in = from && has_col && ra < A_;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (in) {
        const float* p = from + ra * R.sa + bcol * R.sb;
        if (R.sa == 1) {
          const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
          f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w; f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = p[(int64_t)j * R.sa];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) S[n][8 * g + j] = f[j];
    }

  // lam^(i - j) of a diagonal tile of P^T: lane = token i, register 8 s + r = token j = 16 s + 8 h + r; and which are causal
  float diag[kAgg ? 1 : 16];
  uint32_t causal[kAgg ? 1 : 8];
  float li = 0.0f, out0 = 0.0f, out1 = 0.0f;
  if constexpr (!kAgg) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int j = 16 * (r / 8) + 8 * h32 + r % 8;
      diag[r] = j <= l32 ? a.scale * power(l2, (float)(l32 - j)) : 0.0f;
      if (r % 2 == 0) causal[r / 2] = (j <= l32 ? 0xffffu : 0u) | (j + 1 <= l32 ? 0xffff0000u : 0u);
    }
    li = power(l2, (float)l32);
    out0 = R.c_out * power(l2, (float)l32 + e);
    out1 = R.c_out * power(l2, (float)(l32 + 32) + e);
    if (tid < 32) half[tid] = a.scale * power(l2, (float)(32 - tid));
  }

  for (int64_t c = 0; c < nchunk; ++c) {
    int64_t t0;
    const int n = tokens(c, t0);
    if (c) lds_barrier();   // every wave has read the previous chunk
    store_tiles();
    if (tid < kQ && (c == 0 || n < kQ)) into[tid] = tid < n ? R.c_in * power(l2, (float)(n - tid) - e) : 0.0f;
    lds_barrier();
    if (c + 1 < nchunk) load(c + 1);
    if (!live) continue;

    f32x16 y[2] = {};
    if constexpr (!kAgg) {
#pragma unroll
      for (int ks = 0; ks < NS; ++ks) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v0 = S[ks / 2][8 * (ks & 1) + 2 * j], v1 = S[ks / 2][8 * (ks & 1) + 2 * j + 1];
          hi[j] = hi16x2(v0, v1);
          lo[j] = pack_bf16x2(v0 - trunc16(v0), v1 - trunc16(v1));
        }
        const bf16x8 sh = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        const bf16x8 sl = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        const bf16x8 q0 = lds_b8(Qs + l32 * L::kRowQ + 16 * ks + 8 * h32);
        const bf16x8 q1 = lds_b8(Qs + (32 + l32) * L::kRowQ + 16 * ks + 8 * h32);
        y[0] = mfma(sl, q0, y[0]);
        y[1] = mfma(sl, q1, y[1]);
        y[0] = mfma(sh, q0, y[0]);
        y[1] = mfma(sh, q1, y[1]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // the phases' registers do not fit side by side
    const float gone = expm1f((float)n * ld);
    if (gone > -0.5f) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[t][r] = fmaf(S[t][r], gone, S[t][r]);
    } else {
      const float at = power(l2, (float)n);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[t][r] *= at;
    }
    bf16x8 xf[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) xf[ks] = opnd_tr(Vs, L::kRowV, 16 * ks, w * 32, lane);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const float4 w0 = *reinterpret_cast<const float4*>(into + 16 * ks + 8 * h32);
      const float4 w1 = *reinterpret_cast<const float4*>(into + 16 * ks + 8 * h32 + 4);
      const uint4 xv = __builtin_bit_cast(uint4, xf[ks]);
      const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
      const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      uint32_t hi[4], mid[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v0 = bf16_lo(xw[j]) * wt[2 * j], v1 = bf16_hi(xw[j]) * wt[2 * j + 1];
        const float r0 = v0 - trunc16(v0), r1 = v1 - trunc16(v1);
        hi[j] = hi16x2(v0, v1);
        mid[j] = hi16x2(r0, r1);
        lo[j] = hi16x2(r0 - trunc16(r0), r1 - trunc16(r1));
      }
      const bf16x8 xh = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      const bf16x8 xm = __builtin_bit_cast(bf16x8, make_uint4(mid[0], mid[1], mid[2], mid[3]));
      const bf16x8 xl = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 kt = opnd_tr(Ks, L::kRowK, 16 * ks, t * 32, lane);
        S[t] = mfma(kt, xl, S[t]);
        S[t] = mfma(kt, xm, S[t]);
        S[t] = mfma(kt, xh, S[t]);
      }
    }
    if constexpr (!kAgg) {
      __builtin_amdgcn_sched_barrier(0);
      // A NaN or infinity in a token's v makes all of its column's state non-finite, so one state per column tells of
      // it.  It would meet P's zeros in front of the token: it is taken out of V and put back below.
      const bool bad = __ballot(!(fabsf(S[0][0]) < INFINITY)) != 0;
      if (bad) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint4 v = __builtin_bit_cast(uint4, xf[ks]);
          uint32_t xw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((xw[j] & 0x7f80u) == 0x7f80u) xw[j] &= 0xffff0000u;
            if ((xw[j] & 0x7f800000u) == 0x7f800000u) xw[j] &= 0xffffu;
          }
          xf[ks] = __builtin_bit_cast(bf16x8, make_uint4(xw[0], xw[1], xw[2], xw[3]));
        }
      }
      const int o_stride = a.H * R.B;
      const auto ro = make_rsrc(R.o + t0 * o_stride + (int64_t)h * R.B + b0, ((n - 1) * o_stride + cols) * 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int r = 0; r < 16; ++r) y[i][r] *= i ? out1 : out0;
#pragma unroll
        for (int jt = 0; jt <= i; ++jt) {
          __builtin_amdgcn_sched_barrier(0);
          f32x16 m = {};
#pragma unroll
          for (int ks = 0; ks < NS; ++ks)
            m = mfma(lds_b8(Ks + (jt * 32 + turn(l32)) * L::kRowK + 16 * ks + 8 * h32),
                     lds_b8(Qs + (i * 32 + l32) * L::kRowQ + 16 * ks + 8 * h32), m);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float f[8];
            if (jt == i) {
#pragma unroll
              for (int r = 0; r < 8; ++r) f[r] = m[8 * g + r] * diag[8 * g + r];
            } else {
              const float4 w0 = *reinterpret_cast<const float4*>(half + 16 * g + 8 * h32);
              const float4 w1 = *reinterpret_cast<const float4*>(half + 16 * g + 8 * h32 + 4);
              const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
              for (int r = 0; r < 8; ++r) f[r] = m[8 * g + r] * wt[r] * li;
            }
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t mask = jt == i ? causal[4 * g + j] : ~0u;
              ph[j] = hi16x2(f[2 * j], f[2 * j + 1]) & mask;
              pl[j] = pack_bf16x2(f[2 * j] - trunc16(f[2 * j]), f[2 * j + 1] - trunc16(f[2 * j + 1])) & mask;
            }
            y[i] = mfma(xf[2 * jt + g], __builtin_bit_cast(bf16x8, make_uint4(pl[0], pl[1], pl[2], pl[3])), y[i]);
            y[i] = mfma(xf[2 * jt + g], __builtin_bit_cast(bf16x8, make_uint4(ph[0], ph[1], ph[2], ph[3])), y[i]);
          }
        }
        const int tok = i * 32 + l32;
        if (bad) {   // NaN from a non-finite token on
          for (int j = 0; j < 32 * i + 32; ++j) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint4 xv = *reinterpret_cast<const uint4*>(Vs + j * L::kRowV + w * 32 + 16 * g + 8 * h32);
              const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                const float x = r & 1 ? bf16_hi(xw[r / 2]) : bf16_lo(xw[r / 2]);
                y[i][8 * g + r] = fmaf(j <= tok ? x : 0.0f, 0.0f, y[i][8 * g + r]);
              }
            }
          }
        }
        const int row = later ? n - 1 - tok : tok;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int ch = w * 32 + 16 * g + 8 * h32;
          typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
          const u32x4 v = {pack_bf16x2(y[i][8 * g], y[i][8 * g + 1]), pack_bf16x2(y[i][8 * g + 2], y[i][8 * g + 3]),
                           pack_bf16x2(y[i][8 * g + 4], y[i][8 * g + 5]), pack_bf16x2(y[i][8 * g + 6], y[i][8 * g + 7])};
          __builtin_amdgcn_raw_buffer_store_b128(v, ro, ch < cols && tok < n ? (row * o_stride + ch) * 2 : kOut, 0, 0);
        }
      }
    }
  }

  float* to = kAgg ? R.ws + part * row_state + at_head
            : R.to && entry >= 0 && k == (later ? 0 : np - 1) && (nchunk > 0 || !a.seq.slots) ? R.to + entry * row_state + at_head
            : nullptr;
  if (!to || !has_col) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int64_t ra = n * 32 + g * 16 + h32 * 8;
      if (ra >= A_) continue;
      float* p = to + ra * R.sa + bcol * R.sb;
      if (R.sa == 1) {
        *reinterpret_cast<float4*>(p) = make_float4(S[n][8 * g], S[n][8 * g + 1], S[n][8 * g + 2], S[n][8 * g + 3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(S[n][8 * g + 4], S[n][8 * g + 5], S[n][8 * g + 6], S[n][8 * g + 7]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[(int64_t)j * R.sa] = S[n][8 * g + j];
      }
    }
}

// The fold over a cut sequence's pieces: a piece's own state in the workspace becomes the state that enters it.  A
// thread per sequence, role and four elements of the state.
__global__ __launch_bounds__(256) void linear_attention_fold_kernel(LaArgs a) {
  const Role& R = a.role[blockIdx.z];
  const int64_t row_state = (int64_t)a.H * a.KV;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  int64_t s, start, stop;
  if (a.seq.cu) {
    const Run run = find_run<true>(a.seq, blockIdx.y, a.whole);   // whole waves
    if (run.s < 0 || run.k != 0) return;
    s = run.s; start = run.start; stop = run.stop;
  } else {
    s = blockIdx.y; start = s * a.len; stop = start + a.len;
  }
  if (e >= row_state) return;
  const int64_t len = (int64_t)1 << a.shift, n = (stop - start + len - 1) >> a.shift;
  const int64_t v0 = a.seq.cu ? part_of(start >> a.shift, s) : s * n;
  const float ld = a.log_decay[e / a.KV], l2 = ld * 1.4426950408889634f;
  const int64_t entry = a.seq.slots ? seq_slot(a.seq, s) : s;
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  if (R.from && entry >= 0 && (!a.seq.positions || a.seq.positions[s] > 0))
    f = *reinterpret_cast<const float4*>(R.from + entry * row_state + e);
  float4* ws = reinterpret_cast<float4*>(R.ws + v0 * row_state + e);
  const int64_t step = row_state / 4;
  const bool later = R.later != 0;
  const int64_t last = stop - start - (n - 1) * len;   // tokens of the last piece
  for (int64_t i0 = 0; i0 < n; i0 += 8) {
    float4 own[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t k = later ? n - 1 - (i0 + i) : i0 + i;
      own[i] = i0 + i + 1 < n ? ws[k * step] : f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i >= n) break;
      const int64_t k = later ? n - 1 - (i0 + i) : i0 + i;
      ws[k * step] = f;
      const float at = power(l2, (float)(k == n - 1 ? last : len));
      f.x = fmaf(at, f.x, own[i].x);
      f.y = fmaf(at, f.y, own[i].y);
      f.z = fmaf(at, f.z, own[i].z);
      f.w = fmaf(at, f.w, own[i].w);
    }
  }
}

int pad_of(int64_t width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }
int waves_of(int64_t width) { return width <= 64 ? 2 : 4; }
int slabs_of(int64_t width) { return (int)((width + 127) / 128); }

template <int A, int NW, bool kAgg>
hipError_t launch(const LaArgs& a, hipStream_t s) {
  constexpr size_t lds = Lds<A, NW, kAgg>::bytes();
  hipError_t e = hipFuncSetAttribute((const void*)linear_attention_kernel<A, NW, kAgg>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)lds);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.units + 7) / 8 * 8 * a.wgs));
  hipLaunchKernelGGL((linear_attention_kernel<A, NW, kAgg>), grid, dim3(64 * NW), lds, s, a);
  return hipGetLastError();
}

template <bool kAgg>
hipError_t launch_for(int pad, int waves, const LaArgs& a, hipStream_t s) {
  if (waves == 2) return pad == 64 ? launch<64, 2, kAgg>(a, s) : pad == 128 ? launch<128, 2, kAgg>(a, s) : launch<256, 2, kAgg>(a, s);
  return pad == 64 ? launch<64, 4, kAgg>(a, s) : pad == 128 ? launch<128, 4, kAgg>(a, s) : launch<256, 4, kAgg>(a, s);
}

// the roles of `of` (a bit each) that one kernel can take, in one launch; returns what is left
template <bool kAgg>
unsigned launch_some(const LaArgs& all, unsigned of, hipStream_t s, hipError_t* e) {
  LaArgs a = all;
  a.nroles = a.wgs = 0;
  int pad = 0, waves = 0;
  for (int r = 0; r < 3; ++r) {
    if (!(of >> r & 1)) continue;
    const Role& R = all.role[r];
    if (a.nroles && (pad_of(R.A) != pad || waves_of(R.B) != waves)) continue;
    pad = pad_of(R.A);
    waves = waves_of(R.B);
    a.first[a.nroles] = a.wgs;
    a.role[a.nroles++] = R;
    a.wgs += R.slabs;
    of &= ~(1u << r);
  }
  *e = launch_for<kAgg>(pad, waves, a, s);
  return of;
}

void set_shape(Role& R, int64_t A, int64_t B, bool transposed, int64_t K) {
  R.A = (int)A; R.B = (int)B;
  R.sa = transposed ? (int)K : 1;   // the state is (V, K)
  R.sb = transposed ? 1 : (int)K;
  R.slabs = slabs_of(B);
  R.slab = (int)(((B + 31) / 32 + R.slabs - 1) / R.slabs) * 32;
}

}  // namespace

LinearAttentionPlan make_linear_attention_plan(int64_t nseq, int64_t total, int64_t nheads, int64_t kdim, int64_t vdim,
                                               bool packed, int64_t longest, bool backward) {
  LinearAttentionPlan p{};
  const int64_t wgs = nheads * (backward ? 2 * slabs_of(kdim) + slabs_of(vdim) : slabs_of(vdim));
  p.wgs = wgs;
  p.shift = 6;
  while ((int64_t)2 << p.shift <= total / 1024 * wgs + total % 1024 * wgs / 1024) ++p.shift;
  const bool fills = nseq >= (512 + wgs - 1) / wgs;
  if (!packed) {
    const int64_t len = total / nseq;
    p.np = fills || len <= (int64_t)1 << p.shift ? 1 : (len + ((int64_t)1 << p.shift) - 1) >> p.shift;
    p.cut = p.np > 1;
    p.whole = p.shift;
    p.pieces = nseq * p.np;
    p.full = nseq * (p.np - 1);
    p.folds = nseq;
    p.parts = p.cut ? nseq * p.np : 0;
  } else {
    if (longest <= 0 || longest > total) longest = total;
    p.cut = longest > (int64_t)1 << (fills ? p.shift + 2 : p.shift);
    p.whole = fills && (int64_t)2 << p.shift <= total / nseq ? p.shift + 2 : p.shift;
    if (!p.cut) p.shift = p.whole = 62;
    p.np = 1;
    p.pieces = (total >> p.shift) + nseq;
    p.full = total >> p.shift;
    p.folds = total >> p.whole;
    p.parts = p.cut ? (total >> p.shift) + std::min(nseq, total >> p.shift) : 0;
  }
  const size_t one = ((size_t)p.parts * nheads * kdim * vdim * 4 + 255) / 256 * 256;
  p.off_later = one;
  p.ws_total = backward ? 2 * one : one;
  return p;
}

hipError_t launch_linear_attention(const LinearAttentionArgs& p, const LinearAttentionPlan& plan, hipStream_t stream) {
  LaArgs a{};
  a.seq.cu = p.cu; a.seq.slots = p.slots; a.seq.positions = p.positions;
  a.seq.nseq = p.nseq; a.seq.total = p.total; a.seq.nslots = p.nslots;
  a.log_decay = p.log_decay;
  a.len = p.total / p.nseq;
  a.np = (int)plan.np; a.shift = plan.shift; a.whole = plan.whole;
  a.H = (int)p.nheads; a.KV = (int)(p.kdim * p.vdim); a.scale = p.scale;
  const uint16_t *q = static_cast<const uint16_t*>(p.q), *k = static_cast<const uint16_t*>(p.k),
                 *v = static_cast<const uint16_t*>(p.v), *g = static_cast<const uint16_t*>(p.dout);
  const int sq = (int)p.q_stride, sk = (int)p.k_stride, sv = (int)p.v_stride, sg = (int)p.dout_stride;
  float* ws = static_cast<float*>(p.workspace);
  float* ws_later = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + plan.off_later);
  Role fwd{};   // o, or for the gradient only the states
  fwd.q = q; fwd.k = k; fwd.v = v; fwd.q_stride = sq; fwd.k_stride = sk; fwd.v_stride = sv;
  fwd.o = static_cast<uint16_t*>(p.o);
  fwd.from = p.initial_state; fwd.to = p.final_state; fwd.ws = ws;
  fwd.c_out = p.scale; fwd.c_in = 1.0f;
  set_shape(fwd, p.kdim, p.vdim, false, p.kdim);
  Role dv{};
  dv.q = k; dv.k = q; dv.v = g; dv.q_stride = sk; dv.k_stride = sq; dv.v_stride = sg;
  dv.o = static_cast<uint16_t*>(p.dv);
  dv.from = p.d_final_state; dv.to = p.d_initial_state; dv.ws = ws_later;
  dv.later = 1; dv.c_out = 1.0f; dv.c_in = p.scale;
  set_shape(dv, p.kdim, p.vdim, false, p.kdim);
  hipError_t e = hipSuccess;
  if (plan.cut) {
    a.role[0] = fwd;
    a.role[1] = dv;
    a.units = plan.full * p.nheads;
    launch_some<true>(a, p.backward ? 3u : 1u, stream, &e);   // the two have one shape
    if (e != hipSuccess) return e;
    const int64_t blocks = ((int64_t)a.H * a.KV / 4 + 255) / 256;
    hipLaunchKernelGGL(linear_attention_fold_kernel, dim3((unsigned)blocks, (unsigned)plan.folds, p.backward ? 2 : 1), dim3(256), 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.units = plan.pieces * p.nheads;
  if (!p.backward) {
    a.role[0] = fwd;
    launch_some<false>(a, 1u, stream, &e);
    return e;
  }
  Role dq{};
  dq.q = g; dq.k = v; dq.v = k; dq.q_stride = sg; dq.k_stride = sv; dq.v_stride = sk;
  dq.o = static_cast<uint16_t*>(p.dq);
  dq.from = p.initial_state; dq.ws = ws; dq.c_out = p.scale; dq.c_in = 1.0f;
  set_shape(dq, p.vdim, p.kdim, true, p.kdim);
  Role dk{};
  dk.q = v; dk.k = g; dk.v = q; dk.q_stride = sv; dk.k_stride = sg; dk.v_stride = sq;
  dk.o = static_cast<uint16_t*>(p.dk);
  dk.from = p.d_final_state; dk.ws = ws_later; dk.later = 1; dk.c_out = 1.0f; dk.c_in = p.scale;
  set_shape(dk, p.vdim, p.kdim, true, p.kdim);
  a.role[0] = dq;
  a.role[1] = dk;
  a.role[2] = dv;
  for (unsigned left = 7; left && e == hipSuccess;) left = launch_some<false>(a, left, stream, &e);
  return e;
}

}  // namespace mscan
