// api.hip -- C ABI of libmamba_scan (declared in include/mamba_scan.h).
//
// Every entry point validates its arguments on the host before touching the
// HIP runtime; a rejected call launches nothing and returns a status code.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "../../include/mamba_scan.h"
#include "internal.h"

// ---- scratch for the allocation-free forward (mamba_scan_fwd_noalloc) ----
// One array per GPU: each device that loads the library holds its own copy
// until the process ends.  In host code `scratch` names a host-side stand-in,
// not device memory; the device address comes from hipGetSymbolAddress (see
// scratch_address), once per device with that device current, and only that
// address is ever passed to a kernel.
static __device__ __align__(256) unsigned char scratch[MAMBA_SCAN_NOALLOC_SCRATCH_BYTES];

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// A launch of `blocks` workgroups of `threads` work-items: the dispatch's grid size
// counts work-items in 32 bits.
bool launch_ok(int64_t blocks, int64_t threads) {
  int64_t t;
  return blocks >= 0 && mul_ok(blocks, threads, &t) && t <= (int64_t)UINT32_MAX;
}

int check_common(int64_t batch, int64_t dim, int64_t dstate, int io_dtype) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (batch < 1 || dim < 1 || dstate < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (dstate > MAMBA_SCAN_MAX_DSTATE) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  if (!mul_ok(batch, dim, &t) || !mul_ok(t, 64, &t)) return MAMBA_SCAN_ERR_SHAPE;
  return MAMBA_SCAN_OK;
}

int check_fwd_sizes(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype) {
  int st = check_common(batch, dim, dstate, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (seqlen < 0) return MAMBA_SCAN_ERR_SHAPE;
  // a workgroup addresses 64 rows of one tensor with 32-bit byte offsets
  const int64_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (seqlen > 0 && 64 * (seqlen + 8) * esz >= ((int64_t)1 << 31)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  // (batch*dim*(seqlen+64)*4 bytes must be representable)
  if (!mul_ok(batch * dim, seqlen + 64, &t) || !mul_ok(t, 16, &t)) return MAMBA_SCAN_ERR_SHAPE;
  return MAMBA_SCAN_OK;
}

// The forward's launches fit a dispatch: the scan (64-channel groups x time chunks, 512
// work-items), the chunk fix-up (16-channel groups x later chunks x ranges, 128), the carry fold and
// the state copy (one work-item per state).
bool fwd_launches_ok(int64_t batch, int64_t dim, int64_t dstate, const mscan::FwdPlan& p) {
  int64_t t;
  return mul_ok(batch, (dim + 63) / 64, &t) && mul_ok(t, p.nchunks, &t) && launch_ok(t, 512) &&
         mul_ok(batch, (dim + 15) / 16, &t) && mul_ok(t, p.nchunks - 1, &t) && mul_ok(t, p.nranges, &t) &&
         launch_ok(t, 128) &&
         mul_ok(batch * dim, dstate, &t) && launch_ok((t + 255) / 256, 256);
}

// Validation shared by the forward entry points: sizes, flags, pointers and the launch plan.
int check_fwd(const void* u, const void* delta, const float* A_log, const void* B, const void* C, const float* D,
              const void* z, const float* delta_bias, const float* initial_state, const float* final_state,
              const void* y, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype, int flags,
              int64_t nchunks, int states_per_wave, mscan::FwdPlan* plan) {
  int st = check_fwd_sizes(batch, dim, dstate, seqlen, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  // tensors with a seqlen dimension are zero-sized when seqlen == 0 and may then be NULL
  if (!A_log) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && (!u || !delta || !B || !C || !y)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {u, delta, B, C, z, y};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, delta_bias, initial_state, final_state};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  if (!mscan::make_fwd_plan(batch, dim, dstate, seqlen, nchunks, states_per_wave, plan))
    return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!fwd_launches_ok(batch, dim, dstate, *plan)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

int run_fwd(const void* u, const void* delta, const float* A_log, const void* B, const void* C, const float* D,
            const void* z, const float* delta_bias, const float* initial_state, float* final_state, void* y,
            int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype, int flags,
            const mscan::FwdPlan& plan, void* workspace, void* stream) {
  mscan::FwdArgs a{};
  a.u = u; a.delta = delta; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = delta_bias;
  a.h0 = initial_state; a.final_state = final_state; a.y = y;
  a.batch = batch; a.dim = dim; a.dstate = dstate; a.seqlen = seqlen;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  a.workspace = workspace;
  hipError_t e = mscan::launch_fwd(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

// The device address of this GPU's copy of `scratch` (below), looked up once
// per device with that device current.
constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch_addr[kMaxDevices];
std::mutex g_scratch_mu;

hipError_t scratch_address(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  void* p = g_scratch_addr[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch_addr[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
      if (e != hipSuccess) return e;
      if (p == nullptr || !aligned(p, 256)) return hipErrorInvalidSymbol;
      g_scratch_addr[dev].store(p, std::memory_order_release);
    }
  }
  *out = p;
  return hipSuccess;
}

}  // namespace

extern "C" {

const char* mamba_scan_status_str(int status) {
  switch (status) {
    case MAMBA_SCAN_OK: return "ok";
    case MAMBA_SCAN_ERR_NULL: return "a required pointer is NULL";
    case MAMBA_SCAN_ERR_SHAPE: return "a size is out of range";
    case MAMBA_SCAN_ERR_DTYPE: return "io_dtype is not MAMBA_SCAN_F32 or MAMBA_SCAN_BF16";
    case MAMBA_SCAN_ERR_ALIGN: return "a pointer is not aligned to its element size";
    case MAMBA_SCAN_ERR_UNSUPPORTED: return "unsupported option (a size past a documented limit, an unknown flag or an invalid tuning knob)";
    case MAMBA_SCAN_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
    case MAMBA_SCAN_ERR_HIP: return "the HIP runtime reported an error";
    default: return "unknown status";
  }
}

int mamba_scan_abi_version(void) { return MAMBA_SCAN_ABI_VERSION; }

size_t mamba_scan_fwd_workspace_size_ex(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype,
                                        int64_t nchunks, int states_per_wave) {
  if (check_fwd_sizes(batch, dim, dstate, seqlen, io_dtype) != MAMBA_SCAN_OK) return (size_t)-1;
  mscan::FwdPlan p;
  if (!mscan::make_fwd_plan(batch, dim, dstate, seqlen, nchunks, states_per_wave, &p)) return (size_t)-1;
  return p.ws_total;
}

size_t mamba_scan_fwd_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype) {
  return mamba_scan_fwd_workspace_size_ex(batch, dim, dstate, seqlen, io_dtype, 0, 0);
}

int mamba_scan_fwd_ex(const void* u, const void* delta, const float* A_log, const void* B, const void* C,
                      const float* D, const void* z, const float* delta_bias, const float* initial_state,
                      float* final_state, void* y, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                      int io_dtype, int flags, int64_t nchunks, int states_per_wave, void* workspace,
                      size_t workspace_bytes, void* stream) {
  mscan::FwdPlan plan;
  int st = check_fwd(u, delta, A_log, B, C, D, z, delta_bias, initial_state, final_state, y, batch, dim, dstate,
                     seqlen, io_dtype, flags, nchunks, states_per_wave, &plan);
  if (st != MAMBA_SCAN_OK) return st;
  if (plan.ws_total > 0) {
    if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return MAMBA_SCAN_ERR_WORKSPACE;
  }
  return run_fwd(u, delta, A_log, B, C, D, z, delta_bias, initial_state, final_state, y, batch, dim, dstate,
                 seqlen, io_dtype, flags, plan, workspace, stream);
}

int mamba_scan_fwd_noalloc(const void* u, const void* delta, const float* A_log, const void* B, const void* C,
                           const float* D, const void* z, const float* delta_bias, const float* initial_state,
                           float* final_state, void* y, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                           int io_dtype, int flags, void* stream) {
  mscan::FwdPlan plan;
  int st = check_fwd(u, delta, A_log, B, C, D, z, delta_bias, initial_state, final_state, y, batch, dim, dstate,
                     seqlen, io_dtype, flags, 0, 0, &plan);
  if (st != MAMBA_SCAN_OK) return st;
  if (plan.ws_total > (size_t)MAMBA_SCAN_NOALLOC_SCRATCH_BYTES) return MAMBA_SCAN_ERR_WORKSPACE;
  void* ws = nullptr;
  if (plan.ws_total > 0) {
    // everything in the scratch is written before it is read within one call (chunk
    // aggregates, then the carry; the first state group's readout sum), so nothing is cleared
    if (scratch_address(&ws) != hipSuccess) return MAMBA_SCAN_ERR_HIP;
  }
  return run_fwd(u, delta, A_log, B, C, D, z, delta_bias, initial_state, final_state, y, batch, dim, dstate,
                 seqlen, io_dtype, flags, plan, ws, stream);
}

int mamba_scan_fwd(const void* u, const void* delta, const float* A_log, const void* B, const void* C,
                   const float* D, const void* z, const float* delta_bias, const float* initial_state,
                   float* final_state, void* y, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen,
                   int io_dtype, int flags, void* workspace, size_t workspace_bytes, void* stream) {
  return mamba_scan_fwd_ex(u, delta, A_log, B, C, D, z, delta_bias, initial_state, final_state, y, batch, dim,
                           dstate, seqlen, io_dtype, flags, 0, 0, workspace, workspace_bytes, stream);
}

int mamba_scan_fwd_conv(const void* x, const float* conv_weight, const float* conv_bias, const void* conv_state_in,
                        void* conv_state_out, const void* delta, const float* A_log, const void* B, const void* C,
                        const float* D, const void* z, const float* delta_bias, const float* initial_state,
                        float* final_state, void* u_out, void* y, int64_t batch, int64_t dim, int64_t dstate,
                        int64_t seqlen, int io_dtype, int flags, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int st = check_fwd_sizes(batch, dim, dstate, seqlen, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (dstate > 16) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!A_log || !conv_weight) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && (!x || !delta || !B || !C || !y)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {x, delta, B, C, z, y, u_out, conv_state_in, conv_state_out};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, delta_bias, initial_state, final_state, conv_weight, conv_bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  mscan::FwdPlan plan;
  if (!mscan::make_fwd_plan(batch, dim, dstate, seqlen, 0, 0, &plan)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!fwd_launches_ok(batch, dim, dstate, plan)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (plan.ws_total > 0) {
    if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return MAMBA_SCAN_ERR_WORKSPACE;
  }
  mscan::FwdArgs a{};
  a.u = x; a.delta = delta; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = delta_bias;
  a.h0 = initial_state; a.final_state = final_state; a.y = y;
  a.batch = batch; a.dim = dim; a.dstate = dstate; a.seqlen = seqlen;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  a.workspace = workspace;
  a.conv_w = conv_weight; a.conv_b = conv_bias; a.conv_state = conv_state_in; a.u_out = u_out;
  hipError_t e = mscan::launch_fwd(a, plan, static_cast<hipStream_t>(stream));
  if (e == hipSuccess && conv_state_out) {
    // after the scan, which reads conv_state_in (the two may be the same buffer)
    mscan::ConvArgs c{};
    c.x = x; c.state_in = conv_state_in; c.state_out = conv_state_out;
    c.batch = batch; c.dim = dim; c.seqlen = seqlen; c.K = 4; c.io_bf16 = a.io_bf16;
    e = mscan::launch_conv_state(c, static_cast<hipStream_t>(stream));
  }
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

size_t mamba_scan_fwd_varlen_workspace_size(int64_t nseq, int64_t dim, int64_t dstate, int64_t total_len,
                                            int io_dtype) {
  if (nseq < 1) return (size_t)-1;
  if (check_fwd_sizes(1, dim, dstate, total_len, io_dtype) != MAMBA_SCAN_OK) return (size_t)-1;
  mscan::VarlenPlan p;
  if (!mscan::make_varlen_plan(nseq, dim, dstate, total_len, &p)) return (size_t)-1;
  return p.ws_total;
}

int mamba_scan_fwd_varlen(const void* u, const void* delta, const float* A_log, const void* B, const void* C,
                          const float* D, const void* z, const float* delta_bias, const int64_t* cu_seqlens,
                          const float* initial_states, float* final_states, void* y, int64_t nseq, int64_t dim,
                          int64_t dstate, int64_t total_len, int io_dtype, int flags, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (nseq < 1) return MAMBA_SCAN_ERR_SHAPE;
  int st = check_fwd_sizes(1, dim, dstate, total_len, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  mscan::VarlenPlan plan;
  if (!mscan::make_varlen_plan(nseq, dim, dstate, total_len, &plan)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  // grid sizes: the scan's (piece, 64-channel group) items of 512 work-items, the fix-up's
  // (piece, 16-channel group) items of 128
  if (!mul_ok(plan.maxp, (dim + 63) / 64, &t) || !launch_ok(t, 512)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!mul_ok(plan.maxp, (dim + 15) / 16, &t) || !launch_ok(t, 128)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!mul_ok(nseq, dim * dstate, &t) || t > INT32_MAX) return MAMBA_SCAN_ERR_UNSUPPORTED;   // carry threads
  if (!A_log || !cu_seqlens) return MAMBA_SCAN_ERR_NULL;
  if (total_len > 0 && (!u || !delta || !B || !C || !y)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {u, delta, B, C, z, y};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, delta_bias, initial_states, final_states};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  if (!aligned(cu_seqlens, 8)) return MAMBA_SCAN_ERR_ALIGN;
  if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return MAMBA_SCAN_ERR_WORKSPACE;
  mscan::FwdArgs a{};
  a.u = u; a.delta = delta; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = delta_bias;
  a.h0 = initial_states; a.final_state = final_states; a.y = y;
  a.batch = 1; a.dim = dim; a.dstate = dstate; a.seqlen = total_len;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  a.workspace = workspace;
  a.cu = cu_seqlens;
  a.nseq = nseq;
  hipError_t e = mscan::launch_fwd_varlen(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_scan_step(float* state, const void* x, const void* dt, const float* A_log, const void* B, const void* C,
                    const float* D, const void* z, const float* dt_bias, int flags, void* y, int64_t batch,
                    int64_t dim, int64_t dstate, int io_dtype, void* stream) {
  int st = check_common(batch, dim, dstate, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if ((batch + 3) / 4 > 65535) return MAMBA_SCAN_ERR_UNSUPPORTED;   // grid rows of four batch rows
  // a grid row's work-items: 4, 8 or 16 lanes per channel
  if (!launch_ok((dim * (dstate <= 16 ? 4 : dstate <= 32 ? 8 : 16) + 255) / 256, 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!state || !x || !dt || !A_log || !B || !C || !y) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {x, dt, B, C, z, y};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {state, A_log, D, dt_bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  mscan::StepArgs a{};
  a.state = state; a.x = x; a.dt = dt; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = dt_bias;
  a.y = y; a.batch = batch; a.dim = dim; a.dstate = dstate; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  hipError_t e = mscan::launch_step(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

size_t mamba_scan_bwd_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype) {
  if (check_fwd_sizes(batch, dim, dstate, seqlen, io_dtype) != MAMBA_SCAN_OK) return (size_t)-1;
  if (dstate > MAMBA_SCAN_MAX_DSTATE_BWD) return (size_t)-1;
  mscan::BwdPlan p;
  mscan::make_bwd_plan(batch, dim, dstate, seqlen, &p);
  return p.ws_total;
}

int mamba_scan_bwd(const void* u, const void* delta, const float* A_log, const void* B, const void* C,
                   const float* D, const void* z, const float* delta_bias, const float* initial_state,
                   const void* dy, const float* d_final_state, void* du, void* ddelta, float* dA_log, void* dB,
                   void* dC, float* dD, void* dz, float* ddelta_bias, float* d_initial_state, int64_t batch,
                   int64_t dim, int64_t dstate, int64_t seqlen, int io_dtype, int flags, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int st = check_fwd_sizes(batch, dim, dstate, seqlen, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (dstate > MAMBA_SCAN_MAX_DSTATE_BWD) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!A_log || !dA_log) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && (!u || !delta || !B || !C || !dy || !du || !ddelta || !dB || !dC)) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && z && !dz) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {u, delta, B, C, z, dy, du, ddelta, dB, dC, dz};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, delta_bias, initial_state, d_final_state, dA_log, dD, ddelta_bias, d_initial_state};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  mscan::BwdPlan plan;
  mscan::make_bwd_plan(batch, dim, dstate, seqlen, &plan);
  {
    // launches: checkpoint and gradient passes (64-channel groups, 512 work-items), the dB/dC
    // reduction (one per (batch, state, token)), the parameter reduction
    int64_t t, t2;
    if (!mul_ok(batch, (dim + 63) / 64, &t) || !launch_ok(t, 512) || !mul_ok(batch * dstate, seqlen, &t2) ||
        !launch_ok((t2 + 255) / 256, 256) || !launch_ok((dim * dstate + 255) / 256, 256))
      return MAMBA_SCAN_ERR_UNSUPPORTED;
  }
  if (plan.ws_total > 0) {
    if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return MAMBA_SCAN_ERR_WORKSPACE;
  }
  mscan::BwdArgs a{};
  a.u = u; a.delta = delta; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.bias = delta_bias;
  a.h0 = initial_state; a.dy = dy; a.dfs = d_final_state;
  a.du = du; a.ddelta = ddelta; a.dA_log = dA_log; a.dB = dB; a.dC = dC; a.dD = dD; a.dz = dz;
  a.dbias = ddelta_bias; a.dh0 = d_initial_state;
  a.batch = batch; a.dim = dim; a.dstate = dstate; a.seqlen = seqlen;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  a.workspace = workspace;
  hipError_t e = mscan::launch_bwd(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_ssd_fwd(const void* x, const void* dt, const float* A_log, const void* B, const void* C, const float* D,
                  const void* z, const float* dt_bias, const float* initial_state, float* final_state, void* y,
                  int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim, int64_t dstate, int io_dtype,
                  int flags, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (batch < 1 || seqlen < 0 || nheads < 1 || headdim < 1 || dstate < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_UNSUPPORTED;              // bf16 operands only
  if (headdim % 32 != 0 || headdim > 256 || (dstate != 64 && dstate != 128)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  // grid: at most headdim / 32 slices per head, at most 1024 work-items each
  if (!mul_ok(batch, nheads * (headdim / 32), &t) || !launch_ok(t, 1024)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  // a chunk's 64 token rows of x / y (nheads * headdim bf16 each) are addressed with 32-bit offsets
  if (nheads > (1 << 24) / headdim) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!mul_ok(t, seqlen, &t) || !mul_ok(t, headdim * 2, &t)) return MAMBA_SCAN_ERR_SHAPE;
  if (!A_log) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && (!x || !dt || !B || !C || !y)) return MAMBA_SCAN_ERR_NULL;
  const void* v16[] = {x, B, C, z, y, initial_state, final_state};   // 16-byte vector accesses
  for (const void* p : v16)
    if (p && !aligned(p, 16)) return MAMBA_SCAN_ERR_ALIGN;
  if (dt && !aligned(dt, 2)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, dt_bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  mscan::SsdArgs a{};
  a.x = x; a.dt = dt; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.dt_bias = dt_bias;
  a.h0 = initial_state; a.final_state = final_state; a.y = y;
  a.batch = batch; a.seqlen = seqlen; a.nheads = nheads; a.headdim = headdim; a.dstate = dstate;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  hipError_t e = mscan::launch_ssd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_conv1d_fwd(const void* x, const float* weight, const float* bias, const void* conv_state_in,
                     void* conv_state_out, void* u, int64_t batch, int64_t dim, int64_t seqlen, int64_t kernel_size,
                     int io_dtype, int silu, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (batch < 1 || dim < 1 || seqlen < 0) return MAMBA_SCAN_ERR_SHAPE;
  if (kernel_size < 1 || kernel_size > 4) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  if (!mul_ok(batch, dim, &t) || !mul_ok(t, seqlen + 8, &t) || !mul_ok(t, 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  if (!weight) return MAMBA_SCAN_ERR_NULL;
  if (seqlen > 0 && (!x || !u)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {x, u, conv_state_in, conv_state_out};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {weight, bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  mscan::ConvArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.state_in = conv_state_in; a.state_out = conv_state_out; a.u = u;
  a.batch = batch; a.dim = dim; a.seqlen = seqlen; a.K = kernel_size;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.silu = silu != 0;
  hipError_t e = mscan::launch_conv(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

// ---- the SSD layer in serving, and the norm ----

namespace {

int check_ssd_heads(int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups) {
  if (nheads < 1 || headdim < 1 || dstate < 1 || ngroups < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (headdim % 32 != 0 || headdim > 256 || (dstate != 64 && dstate != 128)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (nheads > (1 << 24) / headdim || nheads % ngroups != 0) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

// `rows` tokens of `width` elements, `stride` apart
int check_rows(int64_t rows, int64_t width, int64_t stride) {
  int64_t t;
  if (stride < width || !mul_ok(rows, stride, &t) || !mul_ok(t, 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  return MAMBA_SCAN_OK;
}

// a pool goes with its slots and positions
bool pool_args_ok(const void* pool, const int64_t* slots, const int64_t* positions) {
  return (pool != nullptr) == (slots != nullptr) && (pool != nullptr) == (positions != nullptr);
}

}  // namespace

int mamba_ssd_conv_fwd_varlen(const void* x, const float* weight, const float* bias, const int64_t* cu_seqlens,
                              void* conv_state, const int64_t* slots, const int64_t* positions, void* u, int64_t nseq,
                              int64_t total_len, int64_t width, int64_t kernel_size, int64_t x_stride, int64_t nslots,
                              int io_dtype, int silu, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (nseq < 1 || total_len < 0 || width < 1 || nslots < 0) return MAMBA_SCAN_ERR_SHAPE;
  if (kernel_size < 2 || kernel_size > 4) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int st = check_rows(total_len, width, x_stride);
  if (st != MAMBA_SCAN_OK) return st;
  int64_t t;
  if (!mul_ok(nslots, width, &t) || !mul_ok(t, 16, &t) || !mul_ok(nseq, 32, &t)) return MAMBA_SCAN_ERR_SHAPE;
  // grid: runs of tokens x groups of (at least) 64 channels
  if (!mul_ok((mscan::ssd_conv_runs(nseq, total_len) + 3) / 4, (width + 63) / 64, &t) || !launch_ok(t, 256))
    return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!weight || !cu_seqlens || !pool_args_ok(conv_state, slots, positions)) return MAMBA_SCAN_ERR_NULL;
  if (total_len > 0 && (!x || !u)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {x, u, conv_state};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {weight, bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  const void* i_ptrs[] = {cu_seqlens, slots, positions};
  for (const void* p : i_ptrs)
    if (p && !aligned(p, 8)) return MAMBA_SCAN_ERR_ALIGN;
  if (total_len == 0) return MAMBA_SCAN_OK;
  mscan::SsdConvArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.cu = cu_seqlens; a.conv_state = conv_state; a.slots = slots;
  a.positions = positions; a.u = u; a.nseq = nseq; a.total = total_len; a.width = width; a.x_stride = x_stride;
  a.nslots = nslots; a.K = (int)kernel_size; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16; a.silu = silu != 0;
  hipError_t e = mscan::launch_ssd_conv(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

static int check_ssd_varlen_sizes(int64_t nseq, int64_t total_len, int64_t nheads, int64_t headdim, int64_t dstate,
                                  int64_t ngroups, int64_t max_len, mscan::SsdVarlenPlan* plan) {
  if (nseq < 1 || total_len < 0 || max_len < 0) return MAMBA_SCAN_ERR_SHAPE;
  int st = check_ssd_heads(nheads, headdim, dstate, ngroups);
  if (st != MAMBA_SCAN_OK) return st;
  int64_t t;
  if (nseq > INT32_MAX || !mul_ok(total_len, nheads * headdim, &t) || !mul_ok(t, 4, &t) || t > ((int64_t)1 << 61))
    return MAMBA_SCAN_ERR_SHAPE;
  *plan = mscan::make_ssd_varlen_plan(nseq, total_len, nheads, headdim, dstate, ngroups, max_len);
  // grid: (piece, group of heads, four units of 32 channels), 256 work-items each
  if (!mul_ok(plan->pieces, plan->quads, &t) || !launch_ok(t, 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

size_t mamba_ssd_fwd_varlen_workspace_size(int64_t nseq, int64_t total_len, int64_t nheads, int64_t headdim,
                                           int64_t dstate, int64_t ngroups, int64_t max_len) {
  mscan::SsdVarlenPlan plan;
  if (check_ssd_varlen_sizes(nseq, total_len, nheads, headdim, dstate, ngroups, max_len, &plan) != MAMBA_SCAN_OK) return (size_t)-1;
  return plan.ws_total;
}

int mamba_ssd_fwd_varlen(const void* x, const void* dt, const float* A_log, const void* B, const void* C,
                         const float* D, const void* z, const float* dt_bias, const int64_t* cu_seqlens, float* state,
                         const int64_t* slots, const int64_t* positions, void* y, int64_t nseq, int64_t total_len,
                         int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups, int64_t max_len,
                         int64_t nslots, int64_t x_stride, int64_t dt_stride, int64_t B_stride, int64_t C_stride, int64_t z_stride,
                         int io_dtype, int flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_UNSUPPORTED;   // bf16 operands only
  mscan::SsdVarlenPlan plan;
  int st = check_ssd_varlen_sizes(nseq, total_len, nheads, headdim, dstate, ngroups, max_len, &plan);
  if (st != MAMBA_SCAN_OK) return st;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  if (nslots < 0 || !mul_ok(nslots, nheads * headdim, &t) || !mul_ok(t, dstate * 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  const int64_t inner = nheads * headdim;
  const int64_t widths[] = {inner, nheads, ngroups * dstate, ngroups * dstate, z ? inner : 0};
  const int64_t strides[] = {x_stride, dt_stride, B_stride, C_stride, z ? z_stride : 0};
  for (int i = 0; i < 5; ++i) {
    st = check_rows(total_len, widths[i], strides[i]);
    if (st != MAMBA_SCAN_OK) return st;
    if (strides[i] > (1 << 24)) return MAMBA_SCAN_ERR_UNSUPPORTED;   // a chunk's rows take 32-bit offsets
    if (i != 1 && strides[i] % 8 != 0) return MAMBA_SCAN_ERR_ALIGN;  // 16-byte accesses
  }
  if (!A_log || !cu_seqlens || !pool_args_ok(state, slots, positions)) return MAMBA_SCAN_ERR_NULL;
  if (total_len > 0 && (!x || !dt || !B || !C || !y)) return MAMBA_SCAN_ERR_NULL;
  const void* v16[] = {x, B, C, z, y, state};
  for (const void* p : v16)
    if (p && !aligned(p, 16)) return MAMBA_SCAN_ERR_ALIGN;
  if (dt && !aligned(dt, 2)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, D, dt_bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  const void* i_ptrs[] = {cu_seqlens, slots, positions};
  for (const void* p : i_ptrs)
    if (p && !aligned(p, 8)) return MAMBA_SCAN_ERR_ALIGN;
  if (plan.ws_total > 0) {
    if (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)) return MAMBA_SCAN_ERR_WORKSPACE;
  }
  if (total_len == 0) return MAMBA_SCAN_OK;
  mscan::SsdVarlenArgs a{};
  a.x = x; a.dt = dt; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.z = z; a.dt_bias = dt_bias; a.cu = cu_seqlens;
  a.state = state; a.slots = slots; a.positions = positions; a.y = y; a.nseq = nseq; a.total = total_len;
  a.nslots = nslots; a.nheads = nheads; a.headdim = headdim; a.dstate = dstate; a.ngroups = ngroups;
  a.x_stride = x_stride; a.dt_stride = dt_stride; a.b_stride = B_stride; a.c_stride = C_stride; a.z_stride = z_stride;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  a.workspace = workspace;
  hipError_t e = mscan::launch_ssd_varlen(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_ssd_step(const void* xbc, const void* dt, const float* A_log, const float* conv_weight,
                   const float* conv_bias, void* conv_state, float* state, const int64_t* slots,
                   const int64_t* positions, const float* D, const void* z, const float* dt_bias, void* y,
                   int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate, int64_t ngroups,
                   int64_t kernel_size, int64_t nslots, int64_t xbc_stride, int64_t dt_stride, int64_t z_stride,
                   int io_dtype, int flags, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (batch < 1 || nslots < 0) return MAMBA_SCAN_ERR_SHAPE;
  int st = check_ssd_heads(nheads, headdim, dstate, ngroups);
  if (st != MAMBA_SCAN_OK) return st;
  if (kernel_size < 2 || kernel_size > 4) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (flags & ~(MAMBA_SCAN_FLAG_SOFTPLUS | MAMBA_SCAN_FLAG_EULER)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  const int64_t inner = nheads * headdim, width = inner + 2 * ngroups * dstate;
  int64_t t;
  // grid: slices of at least 8 channels, 256 work-items each
  if (!mul_ok(batch, inner / 8, &t) || !launch_ok(t, 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!mul_ok(nslots, inner, &t) || !mul_ok(t, dstate * 4, &t) || !mul_ok(nslots, width * 16, &t)) return MAMBA_SCAN_ERR_SHAPE;
  st = check_rows(batch, width, xbc_stride);
  if (st == MAMBA_SCAN_OK) st = check_rows(batch, nheads, dt_stride);
  if (st == MAMBA_SCAN_OK && z) st = check_rows(batch, inner, z_stride);
  if (st != MAMBA_SCAN_OK) return st;
  if (!xbc || !dt || !A_log || !conv_weight || !conv_state || !state || !positions || !y) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  const void* io_ptrs[] = {xbc, dt, z, y, conv_state};
  for (const void* p : io_ptrs)
    if (p && !aligned(p, esz)) return MAMBA_SCAN_ERR_ALIGN;
  const void* f_ptrs[] = {A_log, conv_weight, conv_bias, D, dt_bias};
  for (const void* p : f_ptrs)
    if (p && !aligned(p, 4)) return MAMBA_SCAN_ERR_ALIGN;
  if (!aligned(state, 16) || !aligned(positions, 8) || (slots && !aligned(slots, 8))) return MAMBA_SCAN_ERR_ALIGN;
  mscan::SsdStepArgs a{};
  a.xbc = xbc; a.dt = dt; a.A_log = A_log; a.conv_weight = conv_weight; a.conv_bias = conv_bias;
  a.conv_state = conv_state; a.state = state; a.slots = slots; a.positions = positions; a.D = D; a.z = z;
  a.dt_bias = dt_bias; a.y = y; a.batch = batch; a.nslots = nslots; a.xbc_stride = xbc_stride;
  a.dt_stride = dt_stride; a.z_stride = z_stride; a.nheads = (int)nheads; a.headdim = (int)headdim;
  a.dstate = (int)dstate; a.ngroups = (int)ngroups; a.K = (int)kernel_size;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.softplus = (flags & MAMBA_SCAN_FLAG_SOFTPLUS) != 0;
  a.euler = (flags & MAMBA_SCAN_FLAG_EULER) != 0;
  hipError_t e = mscan::launch_ssd_step(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

// sizes and element types shared by the norm and its gradient
static int check_norm(int64_t rows, int64_t dim, int io_dtype, int residual_dtype) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (residual_dtype != io_dtype && residual_dtype != MAMBA_SCAN_F32) return MAMBA_SCAN_ERR_DTYPE;
  if (rows < 0 || dim < 1) return MAMBA_SCAN_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(rows + 1024, dim + 1, &t) || !mul_ok(t, 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  // grids: at most a workgroup per row; 64 work-items a column
  if (!launch_ok(rows, 1024) || !launch_ok((dim + 15) / 16, 1024)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

int mamba_rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps, void* residual_out,
                       void* y, void* scales, float* rstd, int64_t rows, int64_t dim, int io_dtype,
                       int residual_dtype, int out_format, void* stream) {
  int st = check_norm(rows, dim, io_dtype, residual_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (out_format < MAMBA_NORM_OUT_IO || out_format > MAMBA_NORM_OUT_MX8) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!weight || (rows > 0 && (!x || !y || (out_format != MAMBA_NORM_OUT_IO && !scales)))) return MAMBA_SCAN_ERR_NULL;
  if (rows > 0 && (residual == nullptr) != (residual_out == nullptr)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4, rsz = residual_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (!aligned(x, esz) || (out_format == MAMBA_NORM_OUT_IO && !aligned(y, esz)) || !aligned(residual, rsz) ||
      !aligned(residual_out, rsz) || !aligned(weight, 4) || !aligned(rstd, 4) ||
      (out_format == MAMBA_NORM_OUT_ROW8 && !aligned(scales, 4)))
    return MAMBA_SCAN_ERR_ALIGN;
  if (rows == 0) return MAMBA_SCAN_OK;
  mscan::NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out; a.y = y; a.scales = scales;
  a.rstd = rstd; a.rows = rows; a.dim = dim; a.eps = eps; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  a.res_f32 = residual_dtype == MAMBA_SCAN_F32; a.out = out_format;
  hipError_t e = mscan::launch_norm_fwd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

size_t mamba_rms_norm_bwd_workspace_size(int64_t rows, int64_t dim) {
  if (check_norm(rows, dim, MAMBA_SCAN_F32, MAMBA_SCAN_F32) != MAMBA_SCAN_OK) return (size_t)-1;
  return (size_t)(mscan::norm_bwd_parts(rows) * dim) * 4;
}

int mamba_rms_norm_bwd(const void* dy, const void* r, const float* weight, const float* rstd, const void* d_residual,
                       void* dx, float* dresidual, float* dweight, int64_t rows, int64_t dim, int io_dtype,
                       int residual_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_norm(rows, dim, io_dtype, residual_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (dresidual && residual_dtype == io_dtype) return MAMBA_SCAN_ERR_UNSUPPORTED;   // dx is that gradient
  if (!weight || !dweight || (rows > 0 && (!dy || !r || !rstd || !dx))) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4, rsz = residual_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (!aligned(dy, esz) || !aligned(dx, esz) || !aligned(r, rsz) || !aligned(d_residual, rsz) ||
      !aligned(dresidual, 4) || !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dweight, 4))
    return MAMBA_SCAN_ERR_ALIGN;
  const size_t need = mamba_rms_norm_bwd_workspace_size(rows, dim);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return MAMBA_SCAN_ERR_WORKSPACE;
  mscan::NormArgs a{};
  a.x = dy; a.residual = r; a.weight = weight; a.rstd = const_cast<float*>(rstd); a.dres = d_residual; a.y = dx;
  a.residual_out = dresidual; a.dweight = dweight; a.rows = rows; a.dim = dim;
  a.io_bf16 = io_dtype == MAMBA_SCAN_BF16; a.res_f32 = residual_dtype == MAMBA_SCAN_F32; a.workspace = workspace;
  hipError_t e = mscan::launch_norm_bwd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

// ---- linear attention with a fixed decay per head ----

static int check_linear_attention(int64_t nseq, int64_t total_len, int64_t nheads, int64_t kdim, int64_t vdim, bool packed,
                                  int64_t max_len, bool backward, mscan::LinearAttentionPlan* plan) {
  if (nseq < 1 || total_len < 0 || max_len < 0 || nheads < 1 || kdim < 1 || vdim < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (!packed && total_len % nseq != 0) return MAMBA_SCAN_ERR_SHAPE;
  if (kdim % 8 != 0 || vdim % 8 != 0 || kdim > 256 || vdim > 256) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (nheads > (1 << 24) / std::max(kdim, vdim)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  if (nseq > INT32_MAX || !mul_ok(total_len, nheads * std::max(kdim, vdim), &t) || !mul_ok(t, 4, &t) ||
      t > ((int64_t)1 << 61) || !mul_ok(nseq, nheads * kdim, &t) || !mul_ok(t, vdim * 4, &t))
    return MAMBA_SCAN_ERR_SHAPE;
  *plan = mscan::make_linear_attention_plan(nseq, total_len, nheads, kdim, vdim, packed, max_len, backward);
  // grid: a piece's workgroups, heads rounded up to eight at a time, 256 work-items each
  if (!mul_ok(plan->pieces + 8, plan->wgs, &t) || !launch_ok(t, 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

// tokens of an array whose rows take 32-bit offsets and 16-byte accesses
static int check_tokens(const void* p, int64_t total_len, int64_t width, int64_t stride) {
  int st = check_rows(total_len, width, stride);
  if (st != MAMBA_SCAN_OK) return st;
  if (stride > (1 << 24)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (stride % 8 != 0 || !aligned(p, 16)) return MAMBA_SCAN_ERR_ALIGN;
  return total_len > 0 && !p ? MAMBA_SCAN_ERR_NULL : MAMBA_SCAN_OK;
}

static size_t linear_attention_workspace(int64_t nseq, int64_t total_len, int64_t nheads, int64_t kdim, int64_t vdim,
                                         int packed, int64_t max_len, bool backward) {
  mscan::LinearAttentionPlan plan;
  if (check_linear_attention(nseq, total_len, nheads, kdim, vdim, packed != 0, max_len, backward, &plan) != MAMBA_SCAN_OK)
    return (size_t)-1;
  return plan.ws_total;
}

size_t mamba_linear_attention_fwd_workspace_size(int64_t nseq, int64_t total_len, int64_t nheads, int64_t kdim,
                                                 int64_t vdim, int packed, int64_t max_len) {
  return linear_attention_workspace(nseq, total_len, nheads, kdim, vdim, packed, max_len, false);
}

size_t mamba_linear_attention_bwd_workspace_size(int64_t nseq, int64_t total_len, int64_t nheads, int64_t kdim,
                                                 int64_t vdim, int packed, int64_t max_len) {
  return linear_attention_workspace(nseq, total_len, nheads, kdim, vdim, packed, max_len, true);
}

int mamba_linear_attention_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                               const int64_t* cu_seqlens, const float* initial_state, float* final_state,
                               const int64_t* slots, const int64_t* positions, void* o, int64_t nseq, int64_t total_len,
                               int64_t nheads, int64_t kdim, int64_t vdim, int64_t max_len, int64_t nslots,
                               int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, int io_dtype,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_UNSUPPORTED;   // bf16 operands only
  mscan::LinearAttentionPlan plan;
  int st = check_linear_attention(nseq, total_len, nheads, kdim, vdim, cu_seqlens != nullptr, max_len, false, &plan);
  if (st != MAMBA_SCAN_OK) return st;
  if (!(fabsf(scale) < INFINITY)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  if (nslots < 0 || !mul_ok(nslots, nheads * kdim, &t) || !mul_ok(t, vdim * 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  if (!log_decay || (slots && !initial_state && !final_state)) return MAMBA_SCAN_ERR_NULL;
  if (st = check_tokens(q, total_len, nheads * kdim, q_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(k, total_len, nheads * kdim, k_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(v, total_len, nheads * vdim, v_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(o, total_len, nheads * vdim, nheads * vdim); st != MAMBA_SCAN_OK) return st;
  if (!aligned(log_decay, 4) || !aligned(initial_state, 16) || !aligned(final_state, 16) || !aligned(cu_seqlens, 8) ||
      !aligned(slots, 8) || !aligned(positions, 8))
    return MAMBA_SCAN_ERR_ALIGN;
  if (plan.ws_total > 0 && (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)))
    return MAMBA_SCAN_ERR_WORKSPACE;
  if (total_len == 0 && (slots || !final_state)) return MAMBA_SCAN_OK;
  mscan::LinearAttentionArgs a{};
  a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.cu = cu_seqlens; a.initial_state = initial_state;
  a.final_state = final_state; a.slots = slots; a.positions = positions; a.o = o; a.nseq = nseq; a.total = total_len;
  a.nslots = nslots; a.nheads = nheads; a.kdim = kdim; a.vdim = vdim; a.q_stride = q_stride; a.k_stride = k_stride;
  a.v_stride = v_stride; a.scale = scale; a.workspace = workspace;
  hipError_t e = mscan::launch_linear_attention(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_linear_attention_bwd(const void* dout, const void* q, const void* k, const void* v, const float* log_decay,
                               const int64_t* cu_seqlens, const float* initial_state, const float* d_final_state,
                               void* dq, void* dk, void* dv, float* d_initial_state, int64_t nseq, int64_t total_len,
                               int64_t nheads, int64_t kdim, int64_t vdim, int64_t max_len, int64_t do_stride,
                               int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, int io_dtype,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_UNSUPPORTED;
  mscan::LinearAttentionPlan plan;
  int st = check_linear_attention(nseq, total_len, nheads, kdim, vdim, cu_seqlens != nullptr, max_len, true, &plan);
  if (st != MAMBA_SCAN_OK) return st;
  if (!(fabsf(scale) < INFINITY)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!log_decay) return MAMBA_SCAN_ERR_NULL;
  const int64_t inner_k = nheads * kdim, inner_v = nheads * vdim;
  if (st = check_tokens(dout, total_len, inner_v, do_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(q, total_len, inner_k, q_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(k, total_len, inner_k, k_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(v, total_len, inner_v, v_stride); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(dq, total_len, inner_k, inner_k); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(dk, total_len, inner_k, inner_k); st != MAMBA_SCAN_OK) return st;
  if (st = check_tokens(dv, total_len, inner_v, inner_v); st != MAMBA_SCAN_OK) return st;
  if (!aligned(log_decay, 4) || !aligned(initial_state, 16) || !aligned(d_final_state, 16) ||
      !aligned(d_initial_state, 16) || !aligned(cu_seqlens, 8))
    return MAMBA_SCAN_ERR_ALIGN;
  if (plan.ws_total > 0 && (!workspace || workspace_bytes < plan.ws_total || !aligned(workspace, 256)))
    return MAMBA_SCAN_ERR_WORKSPACE;
  if (total_len == 0 && !d_initial_state) return MAMBA_SCAN_OK;
  mscan::LinearAttentionArgs a{};
  a.dout = dout; a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.cu = cu_seqlens; a.initial_state = initial_state;
  a.d_final_state = d_final_state; a.dq = dq; a.dk = dk; a.dv = dv; a.d_initial_state = d_initial_state; a.nseq = nseq;
  a.total = total_len; a.nheads = nheads; a.kdim = kdim; a.vdim = vdim; a.dout_stride = do_stride; a.q_stride = q_stride;
  a.k_stride = k_stride; a.v_stride = v_stride; a.scale = scale; a.workspace = workspace; a.backward = true;
  hipError_t e = mscan::launch_linear_attention(a, plan, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

int mamba_linear_attention_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                                const int64_t* slots, const int64_t* positions, void* o, int64_t batch, int64_t nheads,
                                int64_t kdim, int64_t vdim, int64_t nslots, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, float scale, int io_dtype, void* stream) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (batch < 1 || nslots < 0 || nheads < 1 || kdim < 1 || vdim < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (kdim % 8 != 0 || kdim > 256 || vdim > 256 || nheads > (1 << 24) / std::max(kdim, vdim)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!(fabsf(scale) < INFINITY)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  const int64_t slice = mscan::linear_attention_step_slice(batch, nheads, kdim, vdim);
  if (!mul_ok(batch, nheads * ((vdim + slice - 1) / slice), &t) || !launch_ok(t, 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  if (!mul_ok(nslots, nheads * kdim, &t) || !mul_ok(t, vdim * 4, &t)) return MAMBA_SCAN_ERR_SHAPE;
  int st = check_rows(batch, nheads * kdim, q_stride);
  if (st == MAMBA_SCAN_OK) st = check_rows(batch, nheads * kdim, k_stride);
  if (st == MAMBA_SCAN_OK) st = check_rows(batch, nheads * vdim, v_stride);
  if (st != MAMBA_SCAN_OK) return st;
  if (!q || !k || !v || !log_decay || !state || !positions || !o) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(o, esz) || !aligned(log_decay, 4) ||
      !aligned(state, 16) || !aligned(slots, 8) || !aligned(positions, 8))
    return MAMBA_SCAN_ERR_ALIGN;
  mscan::LinearAttentionStepArgs a{};
  a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.state = state; a.slots = slots; a.positions = positions; a.o = o;
  a.batch = batch; a.nslots = nslots; a.nheads = nheads; a.kdim = kdim; a.vdim = vdim; a.q_stride = q_stride;
  a.k_stride = k_stride; a.v_stride = v_stride; a.scale = scale; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  hipError_t e = mscan::launch_linear_attention_step(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

// ---- norm of groups with an activation ----

static int check_group_norm(int64_t rows, int64_t groups, int64_t width, int io_dtype) {
  if (io_dtype != MAMBA_SCAN_F32 && io_dtype != MAMBA_SCAN_BF16) return MAMBA_SCAN_ERR_DTYPE;
  if (rows < 0 || groups < 1 || width < 1) return MAMBA_SCAN_ERR_SHAPE;
  if (width > 8192 || groups > (1 << 24) / width) return MAMBA_SCAN_ERR_UNSUPPORTED;
  int64_t t;
  // at most a workgroup of 1024 per group, 64 work-items a column
  if (!mul_ok(rows + 2048, groups, &t) || !launch_ok(t, width > 2048 ? 1024 : 256)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  return MAMBA_SCAN_OK;
}

static int check_group_norm_args(int64_t rows, int64_t groups, int64_t width, int64_t z_stride, const void* x, const void* z,
                                 const void* y, const float* weight, const float* bias, float eps, int silu, int io_dtype) {
  int st = check_group_norm(rows, groups, width, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (!(eps >= 0.0f) || (z && silu)) return MAMBA_SCAN_ERR_UNSUPPORTED;
  st = check_rows(rows, groups * width, z ? z_stride : groups * width);
  if (st != MAMBA_SCAN_OK) return st;
  if (rows > 0 && (!x || !y)) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(z, esz) || !aligned(y, esz) || !aligned(weight, 4) || !aligned(bias, 4))
    return MAMBA_SCAN_ERR_ALIGN;
  return MAMBA_SCAN_OK;
}

int mamba_group_norm_fwd(const void* x, const float* weight, const float* bias, const void* z, float eps, void* y,
                         int64_t rows, int64_t groups, int64_t width, int64_t z_stride, int center, int silu, int io_dtype,
                         void* stream) {
  int st = check_group_norm_args(rows, groups, width, z_stride, x, z, y, weight, bias, eps, silu, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (rows == 0) return MAMBA_SCAN_OK;
  mscan::GroupNormArgs a{};
  a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.y = y; a.rows = rows; a.groups = groups; a.width = width;
  a.z_stride = z_stride; a.eps = eps; a.center = center != 0; a.silu = silu != 0; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16;
  hipError_t e = mscan::launch_group_norm_fwd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

size_t mamba_group_norm_bwd_workspace_size(int64_t rows, int64_t groups, int64_t width) {
  if (check_group_norm(rows, groups, width, MAMBA_SCAN_F32) != MAMBA_SCAN_OK) return (size_t)-1;
  return rows == 0 ? 0 : (size_t)(mscan::group_norm_bwd_parts(rows, groups, width) * groups * width) * 8;
}

int mamba_group_norm_bwd(const void* dy, const void* x, const float* weight, const float* bias, const void* z, float eps,
                         void* dx, void* dz, float* dweight, float* dbias, int64_t rows, int64_t groups, int64_t width,
                         int64_t z_stride, int center, int silu, int io_dtype, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int st = check_group_norm_args(rows, groups, width, z_stride, x, z, dx, weight, bias, eps, silu, io_dtype);
  if (st != MAMBA_SCAN_OK) return st;
  if (rows > 0 && (!dy || (z == nullptr) != (dz == nullptr))) return MAMBA_SCAN_ERR_NULL;
  const size_t esz = io_dtype == MAMBA_SCAN_BF16 ? 2 : 4;
  if (!aligned(dy, esz) || !aligned(dz, esz) || !aligned(dweight, 4) || !aligned(dbias, 4)) return MAMBA_SCAN_ERR_ALIGN;
  const size_t need = dweight || dbias ? mamba_group_norm_bwd_workspace_size(rows, groups, width) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return MAMBA_SCAN_ERR_WORKSPACE;
  mscan::GroupNormArgs a{};
  a.dy = dy; a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.y = dx; a.dz = dz; a.dweight = dweight; a.dbias = dbias;
  a.rows = rows; a.groups = groups; a.width = width; a.z_stride = z_stride; a.eps = eps; a.center = center != 0;
  a.silu = silu != 0; a.io_bf16 = io_dtype == MAMBA_SCAN_BF16; a.workspace = workspace;
  hipError_t e = mscan::launch_group_norm_bwd(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? MAMBA_SCAN_OK : MAMBA_SCAN_ERR_HIP;
}

}  // extern "C"
