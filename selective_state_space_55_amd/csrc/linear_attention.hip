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
//
// Mapping.  A workgroup is four waves that walk a piece of one sequence and head; each owns 32 columns of the state (16
// where v has at most 64), all its rows, in MFMA accumulators.  q, k and v of a chunk pass through LDS, the next chunk's
// loads in flight behind them.  A gradient's three products are workgroups of one launch.  The workgroups of eight (sequence,
// head) at a time lie on one XCD each, so that the slabs and products that share q, k, v and do read them from one L2.
//   S^T Q^T  S as bf16 hi + lo (2^-16 of it: one part alone would add an error like o's own rounding), straight from the
//            accumulators: the order of a product's k index is free as long as both operands agree
//   P        formed once a workgroup, a quarter by each wave beside S^T Q^T, whose operands of Q it shares; masked, decayed
//            and passed on through LDS in bf16 hi + lo, as S
//   K^T V    the weighted v in three bf16 parts by truncation (8 bits each: exact), so that a state that leaves keeps fp32's
//            accuracy; in two (2^-16) where none can, in the gradient without an initial state.  K and V by
//            transposing LDS reads
//   S        decays by a factor a chunk whose rounding is carried in 64 bits, so that a head that forgets slowly does not
//            add it up over a long prompt
// 32 columns a wave and A = 128 take 76 KB of LDS and 240 registers: two workgroups on a CU, two waves on a SIMD.
//
// What bounds it: with heads of 128 instruction issue on matrix and vector units.  A wave's chunk of the gradient (128 x
// 128) is 84 MFMAs of 32 cycles, 810 vector instructions and 104 LDS accesses; two waves on a SIMD take 5250 cycles for one
// such chunk each, of which 2690 run MFMAs and 3240 issue vector instructions; a third of these split S and scale it.  8 x
// 2048 tokens, 32 heads of 128 x 128: 349 - 430 us (cards differ), 271 GFLOP of matrix products, 630 - 775 TFLOP/s of
// the 1170 - 1230 that a product of 8192^3 in bf16 reaches.  With heads of 64 HBM: 8 x 2048 tokens, 64 heads, 129 us, 4.2 TB/s.
// 28 sequences of 160 to 4300 tokens, 32 heads of 128: 343 - 410 us, what the longest's chunks take one after another, while
// all of them would fill the GPU for 220; cut, it would wait for a first pass of 100.  One of 20000, 16 heads of 128 x 256, 253 -
// 265 us, of these 92 the pieces' own states, 16 the fold and 179 the main pass (traced); one of 509, 12 heads of 64: 22
// us, eight chunks one after another.  Eight waves of 16 columns on heads of 128, the products interleaved by hand, and keys
// read a product ahead measured the same or worse.
#include "internal.h"
#include "io.h"
#include "mfma.h"
#include "packed.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mscan {
namespace {

constexpr int kQ = 64;   // tokens per chunk

typedef float f32x4 __attribute__((ext_vector_type(4)));
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
  Chunks piece, whole; // a piece; packed sequences of at most `whole` are not cut
  int H, KV;
  int exact;           // a state leaves the call, or may: v goes into it in three parts, else in two
  float scale;
};

__device__ __forceinline__ uint32_t hi16x2(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float trunc16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

__device__ __forceinline__ f32x4 product(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 product(bf16x8 a, bf16x8 b, f32x16 c) { return mfma(a, b, c); }

// makes the compiler wait for a load here
__device__ __forceinline__ void arrived(uint4& v) { asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w)); }

// index m of 32 with bits 2 and 3 exchanged: where operand row m takes row turn(m) of its array, an accumulator's
// registers 8 s .. 8 s + 7 hold the array's rows 16 s + 8 h .. + 7 (h the lane's half), which is an operand's k order
__device__ __forceinline__ int turn(int m) { return (m & 19) | ((m & 4) << 1) | ((m & 8) >> 1); }

// Operands of an MFMA whose k index runs along the rows of a row-major tile, by two transposing reads of 4 rows each; in a
// 16-lane group the lane a + 4 kk addresses row kk and the four columns of a.
// 32x32x16: lane l gets rows k0 + 8 (l / 32) .. + 7 of column n0 + turn(l % 32)
__device__ __forceinline__ bf16x8 opnd32(const uint16_t* base, int pitch, int k0, int n0, int lane) {
  const int g = lane >> 4, m = lane & 15, a = m & 3;
  const uint16_t* p = base + (k0 + 8 * (g >> 1) + (m >> 2)) * pitch + n0 + 16 * (g & 1) + 4 * ((a >> 1) | ((a & 1) << 1));
  const uint2 lo = lds_tr16(p);
  const uint2 hi = lds_tr16(p + 4 * pitch);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}
// 16x16x32: lane l gets rows k0 + 8 (l / 16) .. + 7 of column n0 + step (l % 16 / 4) + l % 4
__device__ __forceinline__ bf16x8 opnd16(const uint16_t* base, int pitch, int k0, int n0, int step, int lane) {
  const uint16_t* p = base + (k0 + 8 * (lane >> 4) + ((lane >> 2) & 3)) * pitch + n0 + step * (lane & 3);
  const uint2 lo = lds_tr16(p);
  const uint2 hi = lds_tr16(p + 4 * pitch);
  return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

__device__ __forceinline__ bf16x8 words(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}

__device__ __forceinline__ float power(float l2, float x) { return x == 0.0f ? 1.0f : __builtin_amdgcn_exp2f(x * l2); }

constexpr int kWaves = 4, kThreads = 64 * kWaves;

// A: width of q and k, rounded up; CW: columns of a wave
template <int A, int CW, bool kAgg>
struct Lds {
  // pitches that spread the rows of one read over the banks
  static constexpr int kRowQ = CW == 32 ? A + 8 : A + 16, kRowK = A + 16, kRowV = kWaves * CW + 16, kRowP = kQ + 8, kRowD = CW + 4;
  static constexpr int kQs = kAgg ? 0 : kQ * kRowQ, kKs = kQ * kRowK, kVs = kQ * kRowV, kPs = kAgg ? 0 : 2 * kQ * kRowP;
  static constexpr size_t bytes() { return 2 * (size_t)(kQs + kKs + kVs + kPs) + 4 * (2 * kQ + (kAgg ? 0 : CW * kRowD)); }
};

__device__ __forceinline__ int64_t part_of(int64_t b, int64_t s) { return b + min(b, s); }

// Workgroups that the tiles leave room for on a CU (160 KB of LDS), which is waves on a SIMD
constexpr int per_cu(int A, int CW) { return A == 256 ? 1 : A == 64 && CW == 16 ? 3 : 2; }

// The sequence that is `rank`-th by length, the longest first, where up to 64 lengths tell, else sequence `rank` (whole waves).
// Workgroups start in this order: 28 sequences of 160 to 4300 tokens, 32 workgroups each, as they come 412 us,
// longest first 400.
__device__ __forceinline__ int64_t by_length(const Packed& p, int64_t rank) {
  if (p.nseq > 64) return rank;
  const int lane = threadIdx.x & 63, n = (int)p.nseq;
  const int at = min(lane, n - 1);
  const int len = (int)max((int64_t)0, min(seq_offset(p, at + 1) - seq_offset(p, at), (int64_t)INT32_MAX));
  int before = 0;
  for (int j = 0; j < n; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    before += other > len || (other == len && j < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(lane < n && before == (int)rank));
}

// kAgg: only the state that a piece would end with from zero
template <int A, int CW, bool kAgg, int kParts>
__global__ __launch_bounds__(kThreads, per_cu(A, CW)) void linear_attention_kernel(LaArgs a) {
  using L = Lds<A, CW, kAgg>;
  constexpr int NB = A / 32;
  extern __shared__ __align__(16) uint16_t sm[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint16_t* Qs = sm;
  uint16_t* Ks = Qs + L::kQs;
  uint16_t* Vs = Ks + L::kKs;
  uint16_t* Ps = Vs + L::kVs;                            // the decayed scores, token i's row: bf16 hi, and kQ rows on the rest
  float* into = reinterpret_cast<float*>(Ps + L::kPs);   // lam^(what follows in the chunk), by token
  float* back = into + kQ;                               // scale lam^(48 - y) by y
  float* diag = back + kQ;                               // scale lam^(i - j) of a diagonal tile, row i
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
    // The main pass takes the sequences' first pieces first, the longest sequence's before the others', and then the pieces
    // that follow them; the other one the pieces that another follows.
    if (!kAgg && number < a.seq.nseq) {
      s = by_length(a.seq, number);
      start = seq_offset(a.seq, s); stop = max(start, seq_offset(a.seq, s + 1)); k = 0;
    } else {
      const Run run = find_run<true>(a.seq, kAgg ? number : number - a.seq.nseq, a.piece);
      if (run.s < 0) return;
      s = run.s; start = run.start; stop = run.stop; k = run.k + (kAgg ? 0 : 1);
    }
    const bool cut = stop - start > a.whole.tokens(1);
    if (!cut && (kAgg || k > 0)) return;
    np = cut ? a.piece.runs(stop - start - 1) + 1 : 1;
    if (k >= np) return;
  } else {
    const int64_t per = kAgg ? a.np - 1 : a.np;
    s = number / per; k = number % per; np = a.np;
    start = s * a.len; stop = start + a.len;
  }
  const bool later = R.later != 0;
  if (kAgg && later) ++k;   // a piece that others precede
  const int64_t t_first = np == 1 ? start : start + a.piece.tokens(k);
  const int64_t t_end = np == 1 ? stop : min(stop, t_first + a.piece.tokens(1));
  const int64_t part = (a.seq.cu ? part_of(a.piece.runs(start), s) : s * np) + k;
  const int nchunk = (int)((t_end - t_first + kQ - 1) / kQ);   // (an array of 2^31 chunks fits no memory)
  const int rest = (int)((t_end - t_first - 1) % kQ) + 1;     // tokens of the last one
  const int A_ = R.A, cols = min(R.slab, R.B - b0);

  const float ld = a.log_decay[h], l2 = ld * 1.4426950408889634f;
  const float e = later ? 0.0f : 1.0f;   // decays between a token's entry and the state that it reads

  auto ld16 = [&](__amdgpu_buffer_rsrc_t r, int off) -> uint4 {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  };
  // a value that the compiler takes as new each time: what is added to it is formed where it is used, not
  // kept in a register over the loop
  auto anew = [](int v) {
    asm volatile("" : "+v"(v));
    return v;
  };

  // Chunks are taken from the first token on, or `later` from the last one back; token i of a chunk in the order they are
  // taken is row i of a tile.  A chunk's descriptor ends with its last token, so that rows past its n tokens, which lie
  // behind the end, or in front of the start at an unsigned offset past it, load as 0.
  constexpr int kCpr = A / 8, kRpp = kThreads / kCpr, kR = kQ / kRpp;   // q, k: 16-byte pieces per row, rows per pass
  constexpr int kVpr = kWaves * CW / 8, kVr = kQ * kVpr / kThreads;     // v
  const int kr = tid / kCpr, kc = (tid % kCpr) * 8;
  const int vr = tid / kVpr, vc = (tid % kVpr) * 8;
  const int out_of = later ? -16 : kOut;   // stays past the end (2^31 - 32 bytes at most) with a chunk's rows added
  const int64_t t_start = later ? t_end - (nchunk == 1 ? rest : kQ) : t_first;
  const uint16_t* kp = R.k + t_start * R.k_stride + (int64_t)h * A_;
  const uint16_t* vp = R.v + t_start * R.v_stride + (int64_t)h * R.B + b0;
  const uint16_t* qp = kAgg ? nullptr : R.q + t_start * R.q_stride + (int64_t)h * A_;
  const int o_stride = a.H * R.B;
  uint16_t* op = kAgg ? nullptr : R.o + t_start * o_stride + (int64_t)h * R.B + b0;
  uint4 qq[kAgg ? 1 : kR], kq[kR], vq[kVr];
  auto load_rows = [&](const uint16_t* base, int stride, int width, int n, int row, int col, int rows, auto& to) {
    const auto r = make_rsrc(base, ((n - 1) * stride + width) * 2);
    const uint32_t step = (later ? -rows : rows) * stride * 2;
    uint32_t off = anew(col < width ? ((later ? n - 1 - row : row) * stride + col) * 2 : out_of);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(to) / 16); ++i) {
      to[i] = ld16(r, (int)off);
      off += step;
    }
  };
  auto load_k = [&](int n, int64_t ahead) {
    kp += ahead * R.k_stride;
    load_rows(kp, R.k_stride, A_, n, kr, kc, kRpp, kq);
  };
  auto load_q = [&](int n, int64_t ahead) {
    if constexpr (!kAgg) {
      qp += ahead * R.q_stride;
      load_rows(qp, R.q_stride, A_, n, kr, kc, kRpp, qq);
    }
  };
  auto load_v = [&](int n, int64_t ahead) {
    vp += ahead * R.v_stride;
    load_rows(vp, R.v_stride, cols, n, vr, vc, kQ / kVr, vq);
  };
  auto store_tiles = [&]() {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      *reinterpret_cast<uint4*>(Ks + (kr + r * kRpp) * L::kRowK + kc) = kq[r];
      if constexpr (!kAgg) *reinterpret_cast<uint4*>(Qs + (kr + r * kRpp) * L::kRowQ + kc) = qq[r];
    }
#pragma unroll
    for (int r = 0; r < kVr; ++r) *reinterpret_cast<uint4*>(Vs + (vr + r * (kQ / kVr)) * L::kRowV + vc) = vq[r];
  };

  if (nchunk > 0) {
    const int n = nchunk == 1 ? rest : kQ;
    load_k(n, 0);
    load_q(n, 0);
    load_v(n, 0);
  }

  // The state: f32x16 tiles of 32 rows x 32 columns, registers 8 s + r row 16 s + 8 (lane / 32) + r of column turn(lane % 32);
  // or pairs of f32x4 tiles of 32 rows x 16 columns, register 4 t + r row 8 (lane / 16) + 4 t + r of column lane % 16.
  // Either way a lane holds eight rows in a row, `step` of these to the next.
  constexpr int kOct = CW == 32 ? 2 * NB : NB, kStep = CW == 32 ? 16 : 32;
  const int wcol = w * CW + (CW == 32 ? turn(lane & 31) : lane & 15);
  const int row8 = 8 * (CW == 32 ? lane >> 5 : lane >> 4);
  const bool has_col = wcol < cols;
  const int64_t entry = a.seq.slots ? seq_slot(a.seq, s) : s;
  const bool started = entry >= 0 && (!a.seq.positions || a.seq.positions[s] > 0);
  const int64_t at_head = (int64_t)h * a.KV, row_state = (int64_t)a.H * a.KV;
  const float* from = kAgg ? nullptr : np > 1 ? R.ws + part * row_state + at_head
                    : R.from && started ? R.from + entry * row_state + at_head : nullptr;
  typedef typename std::conditional<CW == 32, f32x16, f32x4>::type Tile;
  Tile S[CW == 32 ? NB : 2 * NB];
#pragma unroll
  for (int o = 0; o < kOct; ++o) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int ra = o * kStep + row8;
    if (from && has_col && ra < A_) {
      const float* p = from + (int64_t)ra * R.sa + (int64_t)(b0 + wcol) * R.sb;
      if (R.sa == 1) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p), z = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < 4 ? x[j % 4] : z[j % 4];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = p[(int64_t)j * R.sa];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (CW == 32) S[o / 2][8 * (o & 1) + j] = f[j];
      else S[2 * o + j / 4][j % 4] = f[j];
    }
  }
  auto row_of = [&](int o, int j) -> float {
    if constexpr (CW == 32) return S[o / 2][8 * (o & 1) + j];
    else return S[2 * o + j / 4][j % 4];
  };

  float li = 0.0f, out[64 / CW];
  if constexpr (!kAgg) {
    for (int x = tid; x < CW * CW; x += kThreads) diag[x / CW * L::kRowD + x % CW] = a.scale * power(l2, (float)max(x / CW - x % CW, 0));
    li = power(l2, (float)(lane % CW));
#pragma unroll
    for (int i = 0; i < 64 / CW; ++i) out[i] = R.c_out * power(l2, (float)(CW * i + lane % CW) + e);
    if (tid < kQ) back[tid] = a.scale * power(l2, (float)max(48 - tid, 0));
  }

  // The state's decay over a chunk, as a factor whose rounding error goes into the next chunk's, so that a head that forgets
  // slowly does not add it up
  const double whole = exp((double)kQ * (double)ld), part_chunk = exp((double)rest * (double)ld);
  const bool carry = whole > 0x1p-100 && whole < 0x1p100;   // (else the factor has few bits or none)
  const double per_whole = 1.0 / whole;
  double off = 0.0;

  // The loads of the state and of the first chunk end here.  Left in flight into the loop, the state's would make each turn
  // wait at its first use of it, for the next chunk's loads too, and the first chunk's would make the wait for a
  // chunk's loads one for the stores behind them.
#pragma unroll
  for (auto& tile : S) asm volatile("" : "+v"(tile));
#pragma unroll
  for (auto& x : kq) arrived(x);
#pragma unroll
  for (auto& x : vq) arrived(x);
  if constexpr (!kAgg) {
#pragma unroll
    for (auto& x : qq) arrived(x);
  }

  for (int c = 0; c < nchunk; ++c) {
    const int n = c + 1 == nchunk ? rest : kQ;
    if (c) lds_barrier();   // every wave has read the previous chunk
    store_tiles();
    if (tid < kQ && (c == 0 || n < kQ)) into[tid] = tid < n ? R.c_in * power(l2, (float)(n - tid) - e) : 0.0f;
    lds_barrier();
    const int next = c + 2 >= nchunk ? rest : kQ;   // tokens of the next chunk, and how far it is
    const int64_t ahead = later ? -next : kQ;
    const bool more = c + 1 < nchunk;
    if (more) load_k(next, ahead);   // the others follow, so that no wave stands in line for its loads
    const double exactly = (n == kQ ? whole : part_chunk) * (1.0 + off);
    const float fade = (float)exactly;
    off = carry ? (exactly - (double)fade) * per_whole : 0.0;
    Tile y[64 / CW];
    bf16x8 xf[CW == 32 ? 4 : 2];
    {
      const int lc = anew(lane % CW), k8 = anew(8 * (lane / CW));   // an operand's row or column, and its first k
      if constexpr (!kAgg) {
        // S^T Q^T, and the scores, which take the same operands of Q.  A wave's scores: the 32 x 32 tile of token half `pi`
        // by half `pj`, or the 16 x 16 tiles of all tokens by token block w; with the tiles behind their tokens, which
        // come out as zeros, as many for each wave.
        const int pi = CW == 32 ? (0x6 >> w) & 1 : 0, pj = CW == 32 ? w >> 1 : w;
        const uint16_t* const krow = Ks + (CW == 32 ? 32 * pj + turn(lc) : 16 * pj + lc) * L::kRowK + k8;
        Tile score[CW == 32 ? 1 : 4];
#pragma unroll
        for (int o = 0; o < kOct; ++o) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v0 = row_of(o, 2 * j), v1 = row_of(o, 2 * j + 1);
            hi[j] = hi16x2(v0, v1);
            lo[j] = pack_bf16x2(v0 - trunc16(v0), v1 - trunc16(v1));
          }
          const bf16x8 sh = words(hi[0], hi[1], hi[2], hi[3]), sl = words(lo[0], lo[1], lo[2], lo[3]);
          const bf16x8 kf = lds_b8(krow + kStep * o);
          bf16x8 q[64 / CW];
#pragma unroll
          for (int i = 0; i < 64 / CW; ++i) q[i] = lds_b8(Qs + (CW * i + lc) * L::kRowQ + kStep * o + k8);
#pragma unroll
          for (int i = 0; i < 64 / CW; ++i) y[i] = product(sl, q[i], o ? y[i] : Tile{});
          if constexpr (CW == 32) {
            score[0] = product(kf, pi ? q[1] : q[0], o ? score[0] : Tile{});
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) score[i] = product(kf, q[i], o ? score[i] : Tile{});
          }
#pragma unroll
          for (int i = 0; i < 64 / CW; ++i) y[i] = product(sh, q[i], y[i]);
        }
        // decayed, in two bf16 parts.  (No branch here: what a branch skips must not count as the wait for the products.)
#pragma unroll
        for (int x = 0; x < (CW == 32 ? 2 : 4); ++x) {
          const int i = CW == 32 ? pi : x, apart = i - pj, j0 = CW == 32 ? 16 * x + k8 : k8 / 2;   // the lane's first j
          const int last = lc + CW * apart - j0;   // the last register that is not behind the token
          const float* const wt = apart <= 0 ? diag + L::kRowD * lc + j0 : back + 48 - CW * apart + j0;
          const float of = apart <= 0 ? 1.0f : li;
          float f[CW == 32 ? 8 : 4];
#pragma unroll
          for (int r = 0; r < (CW == 32 ? 8 : 4); r += 4) {
            const float4 w4 = *reinterpret_cast<const float4*>(wt + r);
            const float wa[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {   // (bits, not a product: what is behind a token may be a NaN)
              const float m = CW == 32 ? score[0][8 * x + r + u] : score[x][r + u];
              f[r + u] = __uint_as_float(__float_as_uint(m * (wa[u] * of)) & (uint32_t)((r + u - 1 - last) >> 31));
            }
          }
          uint16_t* const p = Ps + (CW * i + lc) * L::kRowP + CW * pj + j0;
          uint32_t ph[CW / 8], pl[CW / 8];
#pragma unroll
          for (int u = 0; u < CW / 8; ++u) {
            ph[u] = hi16x2(f[2 * u], f[2 * u + 1]);
            pl[u] = pack_bf16x2(f[2 * u] - trunc16(f[2 * u]), f[2 * u + 1] - trunc16(f[2 * u + 1]));
          }
          if constexpr (CW == 32) {
            *reinterpret_cast<uint4*>(p) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
            *reinterpret_cast<uint4*>(p + kQ * L::kRowP) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
          } else {
            *reinterpret_cast<uint2*>(p) = make_uint2(ph[0], ph[1]);
            *reinterpret_cast<uint2*>(p + kQ * L::kRowP) = make_uint2(pl[0], pl[1]);
          }
        }
        if (more) load_q(next, ahead);
      }
#pragma unroll
      for (auto& tile : S)
#pragma unroll
        for (int r = 0; r < (CW == 32 ? 16 : 4); ++r) tile[r] *= fade;
#pragma unroll
      for (int ks = 0; ks < kQ / kStep; ++ks) {
        if constexpr (CW == 32) xf[ks] = opnd32(Vs, L::kRowV, 16 * ks, w * 32, lane);
        else xf[ks] = opnd16(Vs, L::kRowV, 32 * ks, w * 16, 4, lane);
        const float4 w0 = *reinterpret_cast<const float4*>(into + kStep * ks + k8);
        const float4 w1 = *reinterpret_cast<const float4*>(into + kStep * ks + k8 + 4);
        const uint4 xv = __builtin_bit_cast(uint4, xf[ks]);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
        const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        uint32_t part3[3][4];   // hi, mid and lo bits of the weighted v
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float v0 = bf16_lo(xw[j]) * wt[2 * j], v1 = bf16_hi(xw[j]) * wt[2 * j + 1];
          const float r0 = v0 - trunc16(v0), r1 = v1 - trunc16(v1);
          part3[0][j] = hi16x2(v0, v1);
          part3[1][j] = kParts == 3 ? hi16x2(r0, r1) : pack_bf16x2(r0, r1);
          if constexpr (kParts == 3) part3[2][j] = hi16x2(r0 - trunc16(r0), r1 - trunc16(r1));
        }
        constexpr int kTiles = sizeof(S) / sizeof(Tile);
        bf16x8 key[2];
#pragma unroll
        for (int b = 0; b < kTiles; b += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (CW == 32) key[u] = opnd32(Ks, L::kRowK, 16 * ks, 32 * (b + u), lane);
            else key[u] = opnd16(Ks, L::kRowK, 32 * ks, 16 * b + 4 * u, 8, lane);
          }
#pragma unroll
          for (int x = kParts - 1; x >= 0; --x)
#pragma unroll
            for (int u = 0; u < 2; ++u) S[b + u] = product(key[u], words(part3[x][0], part3[x][1], part3[x][2], part3[x][3]), S[b + u]);
        }
      }
    }
    // The products' last results are there before any branch: the compiler counts instructions that a branch may skip among
    // those that it waits with (seen in its output; the assembly is tested for it).
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15");
    __builtin_amdgcn_sched_barrier(0);
    if (more) load_v(next, ahead);
    if constexpr (!kAgg) {
      lds_barrier();   // P
      const int lc = anew(lane % CW), k8 = anew(8 * (lane / CW));
      // A NaN or infinity in a token's v makes all of its column's state non-finite, so one state per column tells of
      // it.  It would meet P's zeros in front of the token: it is taken out of V and put back below.
      const bool bad = __ballot(!(fabsf(S[0][0]) < INFINITY)) != 0;
      if (bad) {
#pragma unroll
        for (auto& f : xf) {
          const uint4 v = __builtin_bit_cast(uint4, f);
          uint32_t xw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((xw[j] & 0x7f80u) == 0x7f80u) xw[j] &= 0xffff0000u;
            if ((xw[j] & 0x7f800000u) == 0x7f800000u) xw[j] &= 0xffffu;
          }
          f = words(xw[0], xw[1], xw[2], xw[3]);
        }
      }
      const auto ro = make_rsrc(op, ((n - 1) * o_stride + cols) * 2);
      op += ahead * o_stride;
#pragma unroll
      for (int i = 0; i < 64 / CW; ++i)
#pragma unroll
        for (int r = 0; r < (CW == 32 ? 16 : 4); ++r) y[i][r] *= out[i];
      // + V^T P^T over the tokens up to each tile's last
#pragma unroll
      for (int ks = 0; ks < kQ / kStep; ++ks)
#pragma unroll
        for (int x = 1; x >= 0; --x)
#pragma unroll
          for (int i = 0; i < 64 / CW; ++i) {
            if (CW * (i + 1) <= kStep * ks) continue;
            y[i] = product(xf[ks], lds_b8(Ps + (x * kQ + CW * i + lc) * L::kRowP + kStep * ks + k8), y[i]);
          }
      if (bad) {   // NaN from a non-finite token on
        for (int j = 0; j < kQ; ++j) {
          const uint16_t* v = Vs + j * L::kRowV + w * CW;
#pragma unroll
          for (int r = 0; r < (CW == 32 ? 16 : 4); ++r) {
            const float x = __uint_as_float((uint32_t)v[CW == 32 ? 16 * (r / 8) + k8 + r % 8 : k8 / 2 + r] << 16);
#pragma unroll
            for (int i = 0; i < 64 / CW; ++i) y[i][r] = fmaf(j <= CW * i + lc ? x : 0.0f, 0.0f, y[i][r]);
          }
        }
      }
      typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
      auto store = [&](int tok, int ch, u32x4 v) {
        const int row = later ? n - 1 - tok : tok;
        __builtin_amdgcn_raw_buffer_store_b128(v, ro, ch < cols && tok < n ? (row * o_stride + ch) * 2 : kOut, 0, 0);
      };
      if constexpr (CW == 32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < 2; ++g)
            store(32 * i + lc, w * 32 + 16 * g + k8,
                  u32x4{pack_bf16x2(y[i][8 * g], y[i][8 * g + 1]), pack_bf16x2(y[i][8 * g + 2], y[i][8 * g + 3]),
                        pack_bf16x2(y[i][8 * g + 4], y[i][8 * g + 5]), pack_bf16x2(y[i][8 * g + 6], y[i][8 * g + 7])});
      } else {
        // a lane holds channels 4 g .. + 3 (g = lane / 16) of token 16 i + lane % 16; groups 2 p and 2 p + 1 trade, so that
        // the first has channels 8 p .. + 7 of tile i and the second those of tile i + 1
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16x2(y[i][0], y[i][1]), pack_bf16x2(y[i + 1][0], y[i + 1][1]), false, false);
          const auto z = __builtin_amdgcn_permlane16_swap(pack_bf16x2(y[i][2], y[i][3]), pack_bf16x2(y[i + 1][2], y[i + 1][3]), false, false);
          store(16 * i + 2 * (k8 & 8) + lc, w * 16 + 4 * (k8 >> 3 & 2), u32x4{x[0], z[0], x[1], z[1]});
        }
      }
    }
  }

  float* to = kAgg ? R.ws + part * row_state + at_head
            : R.to && entry >= 0 && k == (later ? 0 : np - 1) && (nchunk > 0 || !a.seq.slots) ? R.to + entry * row_state + at_head
            : nullptr;
  if (!to || !has_col) return;
  const int r8 = anew(row8);
  to += (int64_t)(b0 + anew(wcol)) * R.sb;
#pragma unroll
  for (int o = 0; o < kOct; ++o) {
    const int ra = o * kStep + r8;
    if (ra >= A_) continue;
    float* p = to + (int64_t)ra * R.sa;
    if (R.sa == 1) {
      *reinterpret_cast<f32x4*>(p) = f32x4{row_of(o, 0), row_of(o, 1), row_of(o, 2), row_of(o, 3)};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{row_of(o, 4), row_of(o, 5), row_of(o, 6), row_of(o, 7)};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[(int64_t)j * R.sa] = row_of(o, j);
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
  const int64_t len = a.piece.tokens(1), n = a.piece.runs(stop - start - 1) + 1;
  const int64_t v0 = a.seq.cu ? part_of(a.piece.runs(start), s) : s * n;
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
      own[i] = make_float4(0.f, 0.f, 0.f, 0.f);   // the last one in this order has none
      if (i0 + i + 1 < n) own[i] = ws[k * step];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t k = later ? n - 1 - (i0 + i) : i0 + i;
      if (i0 + i < n) ws[k * step] = f;
      const float at = power(l2, (float)(k == n - 1 ? last : len));
      f.x = fmaf(at, f.x, own[i].x);
      f.y = fmaf(at, f.y, own[i].y);
      f.z = fmaf(at, f.z, own[i].z);
      f.w = fmaf(at, f.w, own[i].w);
    }
  }
}

int pad_of(int64_t width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }
int columns_of(int64_t width) { return width <= 64 ? 16 : 32; }   // of a wave
int slabs_of(int64_t width) { return (int)((width + 127) / 128); }

template <int A, int CW, bool kAgg, int kParts>
hipError_t launch(const LaArgs& a, hipStream_t s) {
  constexpr size_t lds = Lds<A, CW, kAgg>::bytes();
  hipError_t e = hipFuncSetAttribute((const void*)linear_attention_kernel<A, CW, kAgg, kParts>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.units + 7) / 8 * 8 * a.wgs));
  hipLaunchKernelGGL((linear_attention_kernel<A, CW, kAgg, kParts>), grid, dim3(kThreads), lds, s, a);
  return hipGetLastError();
}

template <int CW, bool kAgg, int kParts>
hipError_t launch_pad(int pad, const LaArgs& a, hipStream_t s) {
  return pad == 64 ? launch<64, CW, kAgg, kParts>(a, s) : pad == 128 ? launch<128, CW, kAgg, kParts>(a, s)
                                                                     : launch<256, CW, kAgg, kParts>(a, s);
}

template <bool kAgg>
hipError_t launch_for(int pad, int columns, const LaArgs& a, hipStream_t s) {
  if (columns == 16) return a.exact ? launch_pad<16, kAgg, 3>(pad, a, s) : launch_pad<16, kAgg, 2>(pad, a, s);
  return a.exact ? launch_pad<32, kAgg, 3>(pad, a, s) : launch_pad<32, kAgg, 2>(pad, a, s);
}

// The roles of `of` (a bit each) that one kernel can take, in one launch; returns what is left.  A gradient whose workgroups
// have a CU each takes the widest kernel for all: 6 heads of 64 x 96, 6 and 12 sequences of 217 tokens 24 and 24 us, in
// two launches 31 and 32, but 36 of them 43 and 39; 12 of 512 tokens and 256 x 64 118 and 77.
template <bool kAgg>
unsigned launch_some(const LaArgs& all, unsigned of, hipStream_t s, hipError_t* e) {
  LaArgs a = all;
  a.nroles = a.wgs = 0;
  int pad = 0, columns = 0, wgs = 0;
  for (int r = 0; r < 3; ++r) {
    if (!(of >> r & 1)) continue;
    const Role& R = all.role[r];
    wgs += R.slabs;
    pad = std::max(pad, pad_of(R.A));
    columns = std::max(columns, columns_of(R.B));
  }
  const bool one = a.units * wgs <= 256;
  for (int r = 0; r < 3; ++r) {
    if (!(of >> r & 1)) continue;
    const Role& R = all.role[r];
    if (!one && a.nroles == 0) {
      pad = pad_of(R.A);
      columns = columns_of(R.B);
    }
    if (!one && (pad_of(R.A) != pad || columns_of(R.B) != columns)) continue;
    a.first[a.nroles] = a.wgs;
    a.role[a.nroles++] = R;
    a.wgs += R.slabs;
    of &= ~(1u << r);
  }
  *e = launch_for<kAgg>(pad, columns, a, s);
  return of;
}

void set_shape(Role& R, int64_t A, int64_t B, bool transposed, int64_t K) {
  R.A = (int)A; R.B = (int)B;
  R.sa = transposed ? (int)K : 1;   // the state is (V, K)
  R.sb = transposed ? 1 : (int)K;
  R.slabs = slabs_of(B);
  R.slab = (int)(((B + 15) / 16 + R.slabs - 1) / R.slabs) * 16;
}

}  // namespace

// Sequences are cut only where they leave CUs idle for long enough.  Sequences that do not fill the GPU are cut into the pieces
// that this model finds cheapest: a CU takes `chunk` us for each 64 tokens of a workgroup, two workgroups on it 0.85 of that
// for each (of small heads: two together no more than one), the first pass half of the main one's time, the pieces' states
// are moved at 4.9 TB/s, the fold takes 0.5 us a piece, and launching two more kernels 12 us.  Pieces are as long as one to
// six workgroups a CU share out, and four chunks at least.  Measured, whole, and in pieces of 4, 8, 16 and 32 chunks:
//   2048 tokens of 32 / 64 / 128 workgroups, heads of 128   128  51  67 109 / 125  74  73 114 / 129 137 120 128 (the last in 16)
//   gradients of 2048 tokens of 96 / 192 workgroups         119  82  83 106 / 117 145 125 137
//   8192 tokens of 16 / 64 workgroups, heads of 64          273  42  44  68 118 / 276 109 102  92 126
//   509 tokens of 12 workgroups                              22  29
//   20000 tokens of 32 workgroups, 128 x 256               1193 303 (in 5) 275  272  301, in 20: 242
// Several packed sequences, whose lengths only the device knows, are not cut unless one of the length that the caller bounds
// them by leaves 4096 chunks' time idle (6 of 21 chunks in all, 18 workgroups each: 31 us, cut 40).  Where they fill the GPU
// by themselves, only those over four pieces of a 512th of the work are cut (28 of 32768 tokens, 32 workgroups each: 422 us, with
// those over one piece cut 530).
LinearAttentionPlan make_linear_attention_plan(int64_t nseq, int64_t total, int64_t nheads, int64_t kdim, int64_t vdim,
                                               bool packed, int64_t longest, bool backward) {
  LinearAttentionPlan p{};
  const int64_t wgs = nheads * (backward ? 2 * slabs_of(kdim) + slabs_of(vdim) : slabs_of(vdim));
  p.wgs = wgs;
  if (!packed) longest = total / nseq;
  else if (longest <= 0 || longest > total) longest = total;
  const int64_t most = INT32_MAX, chunks = std::min((longest + kQ - 1) / kQ, most), all = std::min((total + kQ - 1) / kQ, most);
  p.piece = p.whole = most;   // every sequence is one piece, however long it is
  const bool fills = nseq >= (256 + wgs - 1) / wgs;
  if (!fills && (!packed || nseq == 1 || chunks >= (4096 + 255 - nseq * wgs) / (256 - nseq * wgs))) {
    const bool small = kdim <= 64 && vdim <= 64;
    const bool two = backward && (pad_of(kdim) != pad_of(vdim) || columns_of(kdim) != columns_of(vdim));   // launches
    const double chunk = small ? 2.1 : std::max(kdim, vdim) <= 128 ? 3.9 : 7.0;
    const int64_t slots = small ? 512 : 256, fwd = nheads * slabs_of(vdim), rest = wgs - fwd;
    auto rounds = [&](double wgs) { return std::ceil(wgs / slots) * (small || wgs <= slots ? 1.0 : 0.85); };
    double best = (double)chunks * chunk;
    for (int r = 1; r <= 6; ++r) {
      const int64_t want = slots * r / wgs - (packed ? nseq - 1 : 0);
      if (want < 1) continue;
      const int64_t m = std::max<int64_t>(4, ((packed ? all : chunks * nseq) + want - 1) / want);
      if (m >= chunks) continue;
      const double each = (double)((chunks + m - 1) / m), n = packed ? (double)((all + m - 1) / m + nseq - 1) : nseq * each;
      const double us = chunk * m * ((two ? rounds(n * rest) + rounds(n * fwd) : rounds(n * wgs)) +
                                     0.5 * rounds((n - nseq) * (backward ? 2 * fwd : fwd))) +
                        n * nheads * kdim * vdim * (backward ? 24 : 12) / 4.9e6 + each / 2 + 12;
      if (us < best) { best = us; p.piece = m; }
    }
    if (p.piece < most) p.whole = p.piece;
  } else if (fills && packed) {
    const double share = std::max(4.0, (double)all * wgs / 512);
    if (4 * share < chunks) { p.piece = (int64_t)share; p.whole = 4 * p.piece; }
  }
  p.cut = p.piece < most;
  p.np = 1;
  if (!packed) {
    if (p.cut) p.np = (chunks + p.piece - 1) / p.piece;
    p.pieces = nseq * p.np;
    p.full = nseq * (p.np - 1);
    p.folds = nseq;
    p.parts = p.cut ? nseq * p.np : 0;
  } else {
    p.full = p.cut ? total / kQ / p.piece : 0;
    p.pieces = p.full + nseq;
    p.folds = p.cut ? total / kQ / p.whole : 0;
    p.parts = p.cut ? p.full + std::min(nseq, p.full) : 0;
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
  a.np = (int)plan.np; a.piece.n = (uint32_t)plan.piece; a.whole.n = (uint32_t)plan.whole;
  a.H = (int)p.nheads; a.KV = (int)(p.kdim * p.vdim); a.scale = p.scale;
  a.exact = !p.backward || p.d_initial_state;
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
