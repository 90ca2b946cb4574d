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
// Mapping.  A wave owns a unit of 32 channels of a head: its S (N x 32) stays in the wave's
// accumulators, and every product is a 32x32x16 MFMA on bf16 operands with fp32 accumulation.
// A workgroup is four units of one group of heads, which share B, C and B C^T, and a piece of
// one sequence, whose chunks it walks.  The order of an MFMA's k index is free as long as both
// operands agree, so what an accumulator holds (lane = column, rows in runs of four) is an operand
// as it stands, and neither S nor M passes through LDS:
//   S^T C^T  S (lane = channel, k = state, in accumulator order), split into bf16 hi + lo (2^-15 at the most),
//            times C, whose LDS rows are stored in that order
//   M        (B C^T)[j][i], lane = token i, comes from LDS once per workgroup; masked and decayed, it
//            is the right operand of X^T M^T, in bf16 hi + lo as S (one bf16 part alone, 2^-8 of each term, would add
//            an error like that of y's own rounding; the second costs 4% of the time)
//   X, B     as the operands of X^T M^T and of the state update, by transposing LDS reads in
//            accumulator order of the tokens; the scaled x is split into three bf16 parts by
//            truncation (8 bits each: exact), so that the state keeps fp32's accuracy over a long prompt
//   Y        leaves as Y^T: a lane holds four consecutive channels of its token, two lanes
//            trade halves (v_permlane32_swap), and 16 bytes go out per lane
// e^(cum_Q - cum_j) is taken from the sum of the logs behind j, not from a difference of two long
// sums.  73 KB of LDS at N = 128: two workgroups share a CU.
//
// Sequences are cut into pieces that run at once where there are too few sequences and heads to fill
// the GPU: a first pass forms each piece's own state (from zero) and its decay, a fold turns those
// into the state that enters each piece (the associative (a, b) operator), and the main pass
// starts from it.
//
// What bounds it: instruction issue, and waiting for it.  A chunk of a unit (N = 128, gated) is 1280 vector
// instructions (a third of them the splits of S, M and the scaled x; the gate and the epilogue, with 64 exponentials and
// reciprocals at a quarter of the rate, 300), 98 MFMAs of 32 cycles and 126 LDS accesses.  Two waves on a SIMD take
// 18,100 cycles for a chunk each, of which 11,800 issue vector instructions and 6,300 run MFMAs.  Those of two waves
// overlap (two MFMAs beside another wave's 16 multiplies: 91 cycles, apart 64 and 76; 128 for four MFMAs), so neither
// fills the SIMD: 29% of the waves' cycles are waits (B C^T at its barrier, LDS, the chunk's loads).  64 heads, 8 sequences
// of 1024 tokens, a wave per SIMD: 113 us; 16, two waves per SIMD: 179.  A third wave per SIMD would need 168 registers
// (S alone is 64) and 53 KB of LDS.  28 sequences, 32768 tokens, 64 heads of 64, N = 128, gated: 435 - 481 us (cards
// differ), of them the main pass 356 - 385 (1.13 GB; B and C are read again by each XCD), the pieces' own states
// 70, the fold 22; one prompt of 20000 tokens, 32 heads of 128, N = 64: 219 - 241 us; one of 509, 24 heads of 64: 29
// us, three short launches.
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
  int x_stride, dt_stride, b_stride, c_stride, z_stride;
  int shift;          // pieces of 2^shift tokens
  int whole;          // sequences of at most 2^whole tokens are not cut
  float* ws_state;    // (parts, H, P, N): a piece's own state, then the state that enters it
  float* ws_decay;    // (parts, H): sum of log a over a piece
  int H, HP, G;       // heads, head dim, groups
  int nquad;          // workgroups per group of heads
  int softplus, euler;
};

// The workspace's parts of a cut sequence s that starts in block b of 2^shift tokens: one per piece from here
// on.  They end before the next cut sequence's begin, whose block is at least one and as many as there are full
// pieces further; all are below blocks + min(sequences, blocks), so that short sequences take none.
__device__ __forceinline__ int64_t part_of(int64_t b, int64_t s) { return b + min(b, s); }

constexpr float kMild = 32.0f, kLeast = -256.0f;
constexpr int kWaves = 4;   // units of 32 channels per workgroup

template <int N, bool kAgg>
struct Lds {
  static constexpr int kRowB = N + 16;   // pitches that spread the rows of one read over the banks
  static constexpr int kRowC = N + 8;
  static constexpr int kRowX = 40;
  static constexpr int kB = kQ * kRowB, kC = kAgg ? 0 : kQ * kRowC, kX = kQ * kRowX;   // kX: a wave's x tile
  static constexpr int kG = kAgg ? 0 : 3 * 1024;             // the causal tiles of B C^T
  static constexpr int kTerms = kAgg ? kQ : 4 * kQ;          // a wave's 2^(cum_Q - cum) w | cum | wgt | sign of w
  static constexpr size_t bytes() { return 2 * (size_t)(kB + kC + kWaves * kX) + 4 * (size_t)(kG + kWaves * kTerms + kWaves); }
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

// exp(x) - 1 without cancellation: the series up to x^7 below 1/2, where its rest is under 2^-22 of the
// result, and the difference above
__device__ __forceinline__ float expm1_small(float x) {
  float p = fmaf(x, 1.0f / 5040.0f, 1.0f / 720.0f);
  p = fmaf(x, p, 1.0f / 120.0f);
  p = fmaf(x, p, 1.0f / 24.0f);
  p = fmaf(x, p, 1.0f / 6.0f);
  p = fmaf(x, p, 0.5f);
  p = fmaf(x * x, p, x);
  return fabsf(x) < 0.5f ? p : __expf(x) - 1.0f;
}

// kAggregate: only the state that a full piece would end with from zero, and its decay.  Its chunks are
// taken last to first, each token weighted by all that follows it in the piece, until what is left has decayed
// below 2^-kGone (2^-24 of the sum is already past fp32): a head that forgets within a chunk or two reads no more
// than that (28-sequence mix: 70 us, first to last and all of them 96).
constexpr float kGone = 96.0f;
enum Mode { kAggregate, kPlain, kGated };
// kSigned: the input weight w may be negative (Delta without softplus)
template <int N, Mode kMode, bool kSigned>
__global__ __launch_bounds__(256, kMode == kAggregate ? 3 : 2) void ssd_varlen_kernel(VArgs a) {
  constexpr bool kAgg = kMode == kAggregate, kGate = kMode == kGated;
  using L = Lds<N, kAgg>;
  constexpr int NT = N / 32, NS = N / 16;   // S tiles of a unit, k slices over the states
  extern __shared__ __align__(16) uint16_t sm[];
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h32 = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint16_t* Bs = sm;
  uint16_t* Cs = Bs + L::kB;
  uint16_t* Xs = Cs + L::kC + w * L::kX;
  float4* Gs = reinterpret_cast<float4*>(Cs + L::kC + kWaves * L::kX);   // [tile][q][lane]
  float* scl = reinterpret_cast<float*>(Gs) + L::kG + w * L::kTerms;
  float* cum2 = scl + kQ;
  int* gone = reinterpret_cast<int*>(Gs) + L::kG + kWaves * L::kTerms;   // kAgg: waves that need no earlier chunk
  float* wgt = cum2 + kQ;
  uint32_t* sgn = reinterpret_cast<uint32_t*>(wgt + kQ);
  lds_poison(sm, (int)L::bytes());

  // the wave's unit, and the piece
  const int quads = a.G * a.nquad;
  const int64_t number = blockIdx.x / quads;
  const int gk = blockIdx.x % quads, g = gk / a.nquad;
  const int tiles = a.HP / 32, upg = (a.H / a.G) * tiles;   // units per head, per group
  const int ug = (gk % a.nquad) * kWaves + w;
  const bool live = ug < upg;                               // the group's last workgroup may have fewer
  const int u = g * upg + (live ? ug : 0);
  const int h = u / tiles, p0 = (u % tiles) * 32;
  const float rate = -expf(a.A_log[h]), Ah = ssd_held(rate);
  const float A2 = Ah * 1.4426950408889634f, iA = 1.0f / rate;
  const float Dh = a.D ? a.D[h] : 0.0f;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const Packed& q = a.seq;
  const Run run = find_run<kAgg>(q, number, a.shift);
  if (run.s < 0) return;   // no such piece; a sequence without tokens leaves its slot as it is
  const bool cut = run.stop - run.start > (int64_t)1 << a.whole;
  if (!cut && (kAgg || run.k > 0)) return;   // the main pass's first workgroups walk the whole sequence
  const int64_t s = run.s, t_first = run.start + (run.k << a.shift);
  // (no overflow: shift <= 62, t_first 0 .. total)
  const int64_t t_end = cut ? min(run.stop, t_first + ((int64_t)1 << a.shift)) : run.stop;
  const bool last = t_end == run.stop, alone = last && run.k == 0;
  const int64_t v = part_of(run.start >> a.shift, s) + run.k;   // the piece's part of the workspace
  const int64_t nchunk = (t_end - t_first + kQ - 1) / kQ;

  const int64_t unit_state = ((int64_t)h * a.HP + p0) * N, row_state = (int64_t)a.H * a.HP * N;

  const int64_t ch = (int64_t)h * a.HP + p0;
  const uint16_t* Bg = a.B + (int64_t)g * N;
  const uint16_t* Cg = a.C + (int64_t)g * N;
  const int y_stride = a.H * a.HP;

  // Tokens t0 .. t0 + 63 of an array with `stride` elements per token, `width` of which are read: a
  // buffer that ends with the last of them inside the piece, so that loads past it give 0 and
  // stores past it are dropped.
  auto rows = [&](const uint16_t* base, int64_t t0, int stride, int width) {
    const int n = (int)min(t_end - t0, (int64_t)kQ);
    return make_rsrc(base + (n <= 0 ? 0 : t0 * stride), n <= 0 ? 0 : ((n - 1) * stride + width) * 2);
  };
  auto ld16 = [&](__amdgpu_buffer_rsrc_t r, int off) -> uint4 {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  };

  // a value that the compiler takes as new each time: what is added to it is formed where it is used, not
  // kept in a register over the loop
  auto anew = [](int v) {
    asm volatile("" : "+v"(v));
    return v;
  };
  constexpr int kR = kQ * (N / 8) / 256;   // 16-byte pieces of B (and C) per thread, 256 / (N / 8) rows apart
  const int bc_row = tid / (N / 8), bc_col = (tid % (N / 8)) * 8;
  const int b_off = (bc_row * a.b_stride + bc_col) * 2, c_off = (bc_row * a.c_stride + bc_col) * 2;
  const int x_off = ((lane / 4) * a.x_stride + (lane % 4) * 8) * 2;
  uint4 bq[kR], cq[kAgg ? 1 : kR], xq[4];
  uint32_t dtq = 0;
  auto load_bc = [&](int64_t t0) {
    const auto rb = rows(Bg, t0, a.b_stride, N), rc = rows(Cg, t0, a.c_stride, N);
    const int bo = anew(b_off), co = anew(c_off);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      bq[r] = ld16(rb, bo + r * (2048 / N) * a.b_stride * 2);
      if constexpr (!kAgg) cq[r] = ld16(rc, co + r * (2048 / N) * a.c_stride * 2);
    }
  };
  auto load_x = [&](int64_t t0) {
    const auto rx = rows(a.x + ch, t0, a.x_stride, 32);
    const int xo = anew(x_off);
#pragma unroll
    for (int r = 0; r < 4; ++r) xq[r] = ld16(rx, xo + r * 16 * a.x_stride * 2);
    dtq = __builtin_amdgcn_raw_buffer_load_b16(rows(a.dt + h, t0, a.dt_stride, 1), lane * a.dt_stride * 2, 0, 0);
  };
  auto store_tiles = [&]() {
    uint16_t* const bo = Bs + anew(bc_row * L::kRowB + bc_col);
    // states 16 s + {0-3, 8-11 | 4-7, 12-15}: a lane half's eight in one 16-byte read
    uint16_t* const co = Cs + anew(bc_row * L::kRowC + (bc_col & ~15) + (bc_col & 8) / 2);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      *reinterpret_cast<uint4*>(bo + r * (2048 / N) * L::kRowB) = bq[r];
      if constexpr (!kAgg) {
        *reinterpret_cast<uint2*>(co + r * (2048 / N) * L::kRowC) = make_uint2(cq[r].x, cq[r].y);
        *reinterpret_cast<uint2*>(co + r * (2048 / N) * L::kRowC + 8) = make_uint2(cq[r].z, cq[r].w);
      }
    }
    uint16_t* const xo = Xs + anew((lane / 4) * L::kRowX + (lane % 4) * 8);
#pragma unroll
    for (int r = 0; r < 4; ++r) *reinterpret_cast<uint4*>(xo + r * 16 * L::kRowX) = xq[r];
  };
  // Of M_ij = g_ij 2^(cum_i - cum_j) w_j, the factor 2^(r - cum_j) w_j (wgt) is taken into the tile's
  // elements and 2^(cum_i - r) into Y's columns, where r = 0, or for the tile (1, 1) the sum over the first
  // 32 tokens (mid): no exponential per element, and one scaling for S_in^T C^T and both tiles of r = 0.
  // The sums of x M^T then stand 2^kMild higher than y before they are scaled, so x (C.B) w may be that much
  // smaller than fp32's largest number: 2^kMild is the decay over 32 tokens up to which this is done.  Past it
  // (where hardly anything survives 32 tokens) each element takes its own exponential, from wgt = cum_j - log2 w_j.
  // 28-sequence mix: 474 us with 2^96 and 479 with 2^32 (2^64 and 2^48 between them); 20000 tokens 238 and 242.
  float mid = 0.0f;
  bool mild = false;
  // a chunk's decay terms from its dt (later: log2 of the decay behind the chunk, where that is wanted), one token per lane, in powers of two; past the end a = 1 and
  // w = 0.  Returns the sum of log2 a.
  auto decay_terms = [&](int64_t t0, float later) -> float {
    const float r = bf(dtq) + bias;
    float delta = a.softplus ? softplus_log2e(r) * 0.6931471805599453f : r;
    delta = t0 + lane < t_end ? delta : 0.0f;
    // 2^kLeast takes any fp32 state to nothing; a larger decay would only cost the sums behind it their last bits
    const float la = delta * A2, la2 = la < kLeast ? kLeast : la;   // (a NaN stays one)
    const float wj = a.euler || fabsf(delta * Ah) < kTinyStep ? delta : expm1_small(delta * Ah) * iA;
    const float cum = wave_prefix_sum(la2);
    const float rev = wave_prefix_sum(__shfl(la2, 63 - lane));   // from the chunk's end
    const float from = __shfl(rev, 63 - lane);                   // token lane .. the last
    const float next = __shfl_down(from, 1);                     // every lane takes part
    const float behind = lane == 63 ? 0.0f : next;               // lane + 1 .. the last
    scl[lane] = __builtin_amdgcn_exp2f(kAgg ? behind + later : behind) * wj;
    const float end = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cum), 63));
    if constexpr (!kAgg) {
      mid = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cum), 31));
      mild = !kSigned && mid >= -kMild && end - mid >= -kMild;
      cum2[lane] = cum;
      if (mild) {
        wgt[lane] = __builtin_amdgcn_exp2f((lane < 32 ? 0.0f : mid) - cum) * wj;
      } else {
        wgt[lane] = cum - __builtin_amdgcn_logf(fabsf(wj));   // +inf where w = 0
        if constexpr (kSigned) sgn[lane] = __float_as_uint(wj) & 0x80000000u;
      }
    }
    return end;
  };

  // the first chunk's loads, before those that wait for the slot
  load_bc(kAgg ? t_end - kQ : t_first);
  load_x(kAgg ? t_end - kQ : t_first);
  const int64_t slot = kAgg ? -1 : seq_slot(q, s);
  const bool started = slot >= 0 && seq_position(q, s) > 0;
  f32x16 S[NT];
  const float* from = kAgg ? nullptr : !alone ? a.ws_state + v * row_state + unit_state
                    : started ? a.state + slot * row_state + unit_state : nullptr;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from) f = *reinterpret_cast<const float4*>(from + (int64_t)l32 * N + n * 32 + 8 * k + 4 * h32);
      S[n][4 * k] = f.x; S[n][4 * k + 1] = f.y; S[n][4 * k + 2] = f.z; S[n][4 * k + 3] = f.w;
    }

  // rows 8 k + 4 h + {0, 1} and {2, 3} of a diagonal tile that are not behind the lane's column
  uint32_t causal[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int j = 8 * (k / 2) + 2 * (k & 1) + 4 * h32;
    causal[k] = (j <= l32 ? 0xffffu : 0u) | (j + 1 <= l32 ? 0xffff0000u : 0u);
  }

  // (without softplus a decay may grow again)
  auto forgotten = [&](float later) { return a.softplus && later < -kGone; };

  float total = 0.0f;   // log2 of the decay over the chunks so far
  for (int64_t c = 0; c < nchunk; ++c) {
    const int64_t t0 = kAgg ? t_end - (c + 1) * kQ : t_first + c * kQ;
    const int64_t t_next = kAgg ? t0 - kQ : t0 + kQ;
    if (c) lds_barrier();   // every wave has read the previous chunk's B, C and B C^T
    if constexpr (kAgg) {
      if (c && gone[0] + gone[1] + gone[2] + gone[3] == kWaves) break;
    }
    store_tiles();
    const float sum = decay_terms(t0, total);
    total += sum;
    const float at = kAgg ? 1.0f : __builtin_amdgcn_exp2f(sum);
    lds_barrier();
    if (!kAgg || c + 1 < nchunk) load_x(t_next);
    if (kAgg && c + 1 < nchunk) load_bc(t_next);
    uint4 zq[2][2];
    if constexpr (kGate) {
        const auto rz = rows(a.z + ch, t0, a.z_stride, 32);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int zo = (anew(l32) * a.z_stride + 8 * h32 + i * 32 * a.z_stride) * 2;
          zq[i][0] = ld16(rz, zo);
          zq[i][1] = ld16(rz, zo + 32);
        }
      }

    f32x16 y[2] = {};
    if constexpr (!kAgg) {
      // (B C^T) tiles (j, i) = (0, 0), (0, 1), (1, 1), one wave each
      if (w < 3) {
        const uint16_t* br = Bs + ((w == 2) * 32 + l32) * L::kRowB + 4 * h32;
        const uint16_t* cr = Cs + ((w > 0) * 32 + l32) * L::kRowC + 8 * h32;
        f32x16 m = {};
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const uint2 b0 = *reinterpret_cast<const uint2*>(br + 16 * k), b1 = *reinterpret_cast<const uint2*>(br + 16 * k + 8);
          m = mfma(__builtin_bit_cast(bf16x8, make_uint4(b0.x, b0.y, b1.x, b1.y)), lds_b8(cr + 16 * k), m);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) Gs[(w * 4 + k) * 64 + lane] = make_float4(m[4 * k], m[4 * k + 1], m[4 * k + 2], m[4 * k + 3]);
      }
      if (live) {
        // S_in^T C^T over both token tiles
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v0 = S[k / 2][8 * (k & 1) + 2 * j], v1 = S[k / 2][8 * (k & 1) + 2 * j + 1];
            hi[j] = hi16x2(v0, v1);
            lo[j] = pack_bf16x2(v0 - trunc16(v0), v1 - trunc16(v1));
          }
          const bf16x8 sh = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          const bf16x8 sl = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          const bf16x8 c0 = lds_b8(Cs + l32 * L::kRowC + 16 * k + 8 * h32);
          const bf16x8 c1 = lds_b8(Cs + (32 + l32) * L::kRowC + 16 * k + 8 * h32);
#pragma unroll
          for (int r = 0; r < 8; ++r) S[k / 2][8 * (k & 1) + r] *= at;
          y[0] = mfma(sl, c0, y[0]);
          y[1] = mfma(sl, c1, y[1]);
          y[0] = mfma(sh, c0, y[0]);
          y[1] = mfma(sh, c1, y[1]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // the phases' registers do not fit side by side
    bf16x8 xf[4];
    if (live && !(kAgg && forgotten(total - sum))) {
#pragma unroll
      for (int k = 0; k < 4; ++k) xf[k] = opnd_acc_order(Xs, L::kRowX, k, 0, lane);
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
        bf16x8 bt[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) bt[n] = opnd_acc_order(Bs, L::kRowB, k, n * 32, lane);
#pragma unroll
        for (int n = 0; n < NT; ++n) S[n] = mfma(bt[n], xl, S[n]);
#pragma unroll
        for (int n = 0; n < NT; ++n) S[n] = mfma(bt[n], xm, S[n]);
#pragma unroll
        for (int n = 0; n < NT; ++n) S[n] = mfma(bt[n], xh, S[n]);
      }
    }
    if constexpr (kAgg) {
      if (lane == 0) gone[w] = !live || forgotten(total);
    }
    if constexpr (!kAgg) {
      __builtin_amdgcn_sched_barrier(0);
      load_bc(t_next);
      lds_barrier();   // B C^T
      if (!live) continue;
      // A NaN or infinity in a token's x makes all of its channel's state NaN, so one state per channel tells of it.
      // In M's products it would meet the zeros in front of the token; it is taken out of them and put back below.
      const bool bad = __ballot(!(fabsf(S[0][0]) < INFINITY)) != 0;
      if (bad) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 v = __builtin_bit_cast(uint4, xf[k]);
          uint32_t xw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((xw[j] & 0x7f80u) == 0x7f80u) xw[j] &= 0xffff0000u;
            if ((xw[j] & 0x7f800000u) == 0x7f800000u) xw[j] &= 0xffffu;
          }
          xf[k] = __builtin_bit_cast(bf16x8, make_uint4(xw[0], xw[1], xw[2], xw[3]));
        }
      }
      const auto ry = rows(a.y + ch, t0, y_stride, 32);
      const uint16_t* const xrow = Xs + anew(l32 * L::kRowX + 4 * h32);
      const float4* const gl = Gs + anew(lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = i * 32 + l32;
        const float ci = cum2[tok], ei = __builtin_amdgcn_exp2f(ci);
        // + X^T M^T, eight rows of M at a time, in two bf16 parts (all of a tile's at once do not fit the registers); on
        // the diagonal, tokens behind i, whose bits may be anything, become 0
        uint32_t mh[4], ml[4];
        auto add_x = [&](int jb, int k, const float (&f)[4]) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t mask = jb == i ? causal[2 * k + j] : ~0u;
            const float v0 = f[2 * j], v1 = f[2 * j + 1];
            mh[2 * (k & 1) + j] = hi16x2(v0, v1) & mask;
            ml[2 * (k & 1) + j] = pack_bf16x2(v0 - trunc16(v0), v1 - trunc16(v1)) & mask;
          }
          if (k & 1) {
            y[i] = mfma(xf[2 * jb + k / 2], __builtin_bit_cast(bf16x8, make_uint4(ml[0], ml[1], ml[2], ml[3])), y[i]);
            y[i] = mfma(xf[2 * jb + k / 2], __builtin_bit_cast(bf16x8, make_uint4(mh[0], mh[1], mh[2], mh[3])), y[i]);
          }
        };
        if (mild) {
          auto tile = [&](int jb, float each) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 gv = gl[((i + jb) * 4 + k) * 64];
              const float4 wj = *reinterpret_cast<const float4*>(wgt + jb * 32 + 8 * k + 4 * h32);
              float f[4] = {gv.x * wj.x, gv.y * wj.y, gv.z * wj.z, gv.w * wj.w};
              if (jb) {
#pragma unroll
                for (int r = 0; r < 4; ++r) f[r] *= each;
              }
              add_x(jb, k, f);
            }
          };
          tile(0, 1.0f);
#pragma unroll
          for (int r = 0; r < 16; ++r) y[i][r] *= ei;
          if (i) tile(1, __builtin_amdgcn_exp2f(ci - mid));
        } else {
#pragma unroll
          for (int r = 0; r < 16; ++r) y[i][r] *= ei;
#pragma unroll
          for (int jb = 0; jb <= i; ++jb) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j0 = jb * 32 + 8 * k + 4 * h32;
              const float4 gv = gl[((i + jb) * 4 + k) * 64];
              const float4 cj = *reinterpret_cast<const float4*>(wgt + j0);
              const float ga[4] = {gv.x, gv.y, gv.z, gv.w}, cja[4] = {cj.x, cj.y, cj.z, cj.w};
              float f[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) f[r] = ga[r] * __builtin_amdgcn_exp2f(ci - cja[r]);
              if constexpr (kSigned) {
                const uint4 sj = *reinterpret_cast<const uint4*>(sgn + j0);
                const uint32_t sa[4] = {sj.x, sj.y, sj.z, sj.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) f[r] = __uint_as_float(__float_as_uint(f[r]) ^ sa[r]);
              }
              add_x(jb, k, f);
            }
          }
        }
        if (bad) {   // NaN from a non-finite token on
          for (int j = 0; j < 32 * i + 32; ++j) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint2 xv = *reinterpret_cast<const uint2*>(Xs + j * L::kRowX + 4 * h32 + 8 * k);
              const float xj[4] = {bf16_lo(xv.x), bf16_hi(xv.x), bf16_lo(xv.y), bf16_hi(xv.y)};
#pragma unroll
              for (int r = 0; r < 4; ++r) y[i][4 * k + r] = fmaf(j <= tok ? xj[r] : 0.0f, 0.0f, y[i][4 * k + r]);
            }
          }
        }
        // + D x, gate, and out: channels 8 k + 4 h .. + 3 of the lane's token
        uint32_t zw[8] = {zq[i][0].x, zq[i][0].y, zq[i][0].z, zq[i][0].w, zq[i][1].x, zq[i][1].y, zq[i][1].z, zq[i][1].w};
        if constexpr (kGate) {
          swap32(zw[0], zw[2]);
          swap32(zw[1], zw[3]);
          swap32(zw[4], zw[6]);
          swap32(zw[5], zw[7]);
        }
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint2 xv = *reinterpret_cast<const uint2*>(xrow + i * 32 * L::kRowX + 8 * k);
          const uint32_t xw[2] = {xv.x, xv.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v0 = fmaf(Dh, bf16_lo(xw[j]), y[i][4 * k + 2 * j]), v1 = fmaf(Dh, bf16_hi(xw[j]), y[i][4 * k + 2 * j + 1]);
            if constexpr (kGate) {
              v0 *= silu(bf16_lo(zw[2 * k + j]));
              v1 *= silu(bf16_hi(zw[2 * k + j]));
            }
            o[2 * k + j] = pack_bf16x2(v0, v1);
          }
        }
        const int yo = (anew(l32) * y_stride + 8 * h32 + i * 32 * y_stride) * 2;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          swap32(o[4 * k], o[4 * k + 2]);
          swap32(o[4 * k + 1], o[4 * k + 3]);
          typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]}, ry, yo + 32 * k, 0, 0);
        }
      }
    }
  }

  if (!live) return;
  float* to = kAgg ? a.ws_state + v * row_state + unit_state
            : last && slot >= 0 ? a.state + slot * row_state + unit_state : nullptr;
  if (kAgg && lane == 0 && p0 == 0) a.ws_decay[v * a.H + h] = total;
  if (!to) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<float4*>(to + (int64_t)l32 * N + n * 32 + 8 * k + 4 * h32) =
          make_float4(S[n][4 * k], S[n][4 * k + 1], S[n][4 * k + 2], S[n][4 * k + 3]);
}

// The fold over a sequence's pieces: entry k of its part of ws_state, piece k's own state, becomes the
// state that enters piece k.  A thread per cut sequence and four states; a cut sequence is found by the number
// of its first run of 2^whole tokens among the full ones, so that the grid does not grow with the uncut ones.
__global__ __launch_bounds__(256) void ssd_fold_kernel(VArgs a, int N) {
  const Packed& q = a.seq;
  const uint32_t row_state = (uint32_t)a.H * a.HP * N;   // at most 2^24 channels x 128 states
  const uint32_t e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const bool in = e < row_state;   // (whole waves look for the sequence)
  const int h = (int)(e / (uint32_t)(a.HP * N));
  const Run run = find_run<true>(q, blockIdx.y, a.whole);
  if (run.s < 0 || run.k != 0) return;
  const int64_t s = run.s, v0 = part_of(run.start >> a.shift, s), slot = seq_slot(q, s);
  const int64_t n = (run.stop - run.start + ((int64_t)1 << a.shift) - 1) >> a.shift;
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  if (slot >= 0 && seq_position(q, s) > 0 && in) f = *reinterpret_cast<const float4*>(a.state + slot * row_state + e);
  if (!in) return;
  float4* ws = reinterpret_cast<float4*>(a.ws_state + v0 * row_state + e);
  const int64_t step = row_state / 4;
  const float* decay = a.ws_decay + v0 * a.H + h;
  // the last piece has no state of its own; eight at a time, so that a short chain costs one trip to memory
  for (int64_t k0 = 0; k0 < n; k0 += 8) {
    float4 own[8];
    float at[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      own[k] = k0 + k + 1 < n ? ws[(k0 + k) * step] : f;
      at[k] = k0 + k + 1 < n ? exp2f(decay[(k0 + k) * a.H]) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k0 + k < n) ws[(k0 + k) * step] = f;
      f.x = fmaf(at[k], f.x, own[k].x);
      f.y = fmaf(at[k], f.y, own[k].y);
      f.z = fmaf(at[k], f.z, own[k].z);
      f.w = fmaf(at[k], f.w, own[k].w);
    }
  }
}

template <int N, Mode kMode, bool kSigned>
hipError_t launch(const VArgs& a, dim3 grid, hipStream_t s) {
  constexpr size_t lds = Lds<N, kMode == kAggregate>::bytes();
  hipError_t e = hipFuncSetAttribute((const void*)ssd_varlen_kernel<N, kMode, kSigned>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((ssd_varlen_kernel<N, kMode, kSigned>), grid, dim3(256), lds, s, a);
  return hipGetLastError();
}

template <int N>
hipError_t run(const VArgs& a, const SsdVarlenPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.pieces * p.quads));
  if (p.cut) {
    const unsigned full = (unsigned)(a.seq.total >> a.shift);   // pieces that another one follows, at most
    hipError_t e = launch<N, kAggregate, true>(a, dim3((unsigned)(full * p.quads)), s);
    if (e != hipSuccess) return e;
    const int64_t blocks = ((int64_t)a.H * a.HP * N / 4 + 255) / 256;
    hipLaunchKernelGGL(ssd_fold_kernel, dim3((unsigned)blocks, (unsigned)(a.seq.total >> a.whole)), dim3(256), 0, s, a, N);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.softplus) return a.z ? launch<N, kGated, false>(a, grid, s) : launch<N, kPlain, false>(a, grid, s);
  return a.z ? launch<N, kGated, true>(a, grid, s) : launch<N, kPlain, true>(a, grid, s);
}

// workgroups of a group's units
int64_t quads_of(int64_t nheads, int64_t headdim, int64_t ngroups) { return (nheads / ngroups * (headdim / 32) + kWaves - 1) / kWaves; }

}  // namespace

// Pieces: as many tokens as share them out over two rounds of two workgroups per CU, a power of two
// (so that a piece number needs no division).  32768 tokens of 28 sequences, 32 workgroups a piece: 479 us in
// pieces of 1024, 471 in 512, 536 in 2048; 20000 tokens of one sequence, 32 a piece: 240 us in 512, 268 in 256,
// 255 in 1024; 509 tokens, 12 workgroups a piece: 29 us in 64, 32 in 128, 45 in 256.
// Where the sequences fill the GPU by themselves, those of up to four pieces are better left whole if they are all like
// that: the host knows it from the hint and launches the main pass alone (16 sequences of 256 tokens, 32 workgroups
// each: 55 us whole, 105 in pieces of 128).  Without a hint a mean of two pieces or more says so, but bounds no
// sequence: the launches for the cut ones are there and the device cuts those over four pieces (the 16 of 256: 68
// us; 28 sequences with one of 50000 tokens among 60000 770 us, left whole 4448).  With shorter means a sequence of four
// pieces would outlast all others: every sequence over one piece is cut (32768 tokens of 28 sequences of 120 to 3600: 490 us,
// with those of up to four pieces whole 571).
SsdVarlenPlan make_ssd_varlen_plan(int64_t nseq, int64_t total, int64_t nheads, int64_t headdim, int64_t dstate,
                                   int64_t ngroups, int64_t longest) {
  SsdVarlenPlan p{};
  p.quads = quads_of(nheads, headdim, ngroups) * ngroups;
  p.shift = 6;
  while ((int64_t)2 << p.shift <= total / 1024 * p.quads + total % 1024 * p.quads / 1024) ++p.shift;
  const bool fills = nseq >= (512 + p.quads - 1) / p.quads;
  if (longest <= 0 || longest > total) longest = total;
  p.cut = longest > (int64_t)1 << (fills ? p.shift + 2 : p.shift);
  p.whole = fills && (int64_t)2 << p.shift <= total / nseq ? p.shift + 2 : p.shift;
  if (!p.cut) p.shift = p.whole = 62;   // every sequence is one piece, however long it is
  p.pieces = (total >> p.shift) + nseq;   // piece numbers end below that
  if (p.cut) {
    const size_t parts = (size_t)((total >> p.shift) + std::min(nseq, total >> p.shift));
    p.off_decay = (parts * nheads * headdim * dstate * 4 + 255) / 256 * 256;
    p.ws_total = p.off_decay + (parts * nheads * 4 + 255) / 256 * 256;
  }
  return p;
}

hipError_t launch_ssd_varlen(const SsdVarlenArgs& p, const SsdVarlenPlan& plan, hipStream_t stream) {
  VArgs a{};
  a.seq.cu = p.cu; a.seq.slots = p.slots; a.seq.positions = p.positions;
  a.seq.nseq = p.nseq; a.seq.total = p.total; a.seq.nslots = p.nslots;
  a.x = static_cast<const uint16_t*>(p.x); a.dt = static_cast<const uint16_t*>(p.dt); a.A_log = p.A_log;
  a.B = static_cast<const uint16_t*>(p.B); a.C = static_cast<const uint16_t*>(p.C); a.D = p.D;
  a.z = static_cast<const uint16_t*>(p.z); a.dt_bias = p.dt_bias; a.state = p.state; a.y = static_cast<uint16_t*>(p.y);
  a.x_stride = (int)p.x_stride; a.dt_stride = (int)p.dt_stride; a.b_stride = (int)p.b_stride;
  a.c_stride = (int)p.c_stride; a.z_stride = (int)p.z_stride;
  a.H = (int)p.nheads; a.HP = (int)p.headdim; a.G = (int)p.ngroups; a.softplus = p.softplus; a.euler = p.euler;
  a.nquad = (int)(plan.quads / p.ngroups);
  a.shift = plan.shift;
  a.whole = plan.whole;
  if (plan.cut) {
    a.ws_state = static_cast<float*>(p.workspace);
    a.ws_decay = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + plan.off_decay);
  }
  return p.dstate == 128 ? run<128>(a, plan, stream) : run<64>(a, plan, stream);
}

}  // namespace mscan
