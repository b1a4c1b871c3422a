// C-ABI layer of the SSD scan's gradients (declared in include/mamba2_ssd.h):
// argument validation before any HIP call.
#include "../../include/mamba2_ssd.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "ssd_bwd_internal.h"

namespace {

using namespace mscan::api;

constexpr int64_t kMaxStride = int64_t{1} << 24;

int check_dims(int32_t batch, int32_t seqlen, int32_t nheads, int32_t headdim, int32_t d_state, int32_t ngroups,
               int32_t io_dtype) {
  if (batch < 1 || seqlen < 1 || nheads < 1 || ngroups < 1)
    return fail(MAMBA_ERR_SHAPE, "dims must be >= 1 (batch=%d seqlen=%d nheads=%d ngroups=%d)", batch, seqlen, nheads,
                ngroups);
  if (headdim != 64) return fail(MAMBA_ERR_SHAPE, "headdim must be 64 (got %d)", headdim);
  if (d_state != 64 && d_state != 128) return fail(MAMBA_ERR_SHAPE, "d_state must be 64 or 128 (got %d)", d_state);
  if (nheads % ngroups != 0) return fail(MAMBA_ERR_SHAPE, "ngroups (%d) must divide nheads (%d)", ngroups, nheads);
  if (batch > 65535 || nheads > 65535)
    return fail(MAMBA_ERR_SHAPE, "batch and nheads must be <= 65535 (got %d, %d)", batch, nheads);
  if (!below_2_31({batch, seqlen, nheads, headdim}) || !below_2_31({batch, seqlen, ngroups, d_state}))
    return fail(MAMBA_ERR_SHAPE, "tensor too large (batch*seqlen*nheads*headdim must be < 2^31)");
  if (io_dtype != MAMBA_F32 && io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_DTYPE, "io_dtype must be MAMBA_F32 (0) or MAMBA_BF16 (1), got %d", io_dtype);
  return MAMBA_OK;
}

// An io input whose rows (batch, step) are `stride` elements apart.
struct Rows {
  const char* name;
  const void* p;
  int64_t stride, width;
  size_t align;
};

}  // namespace

extern "C" {

size_t mamba2_ssd_bwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t headdim, int32_t d_state,
                                      int32_t ngroups, int32_t io_dtype) {
  const std::string saved = last_error();
  const int st = check_dims(batch, seqlen, nheads, headdim, d_state, ngroups, io_dtype);
  last_error() = saved;
  return st ? 0 : mscan::ssd_bwd_ws_bytes(batch, seqlen, nheads, d_state, ngroups);
}

int mamba2_ssd_bwd(int32_t batch, int32_t seqlen, int32_t nheads, int32_t headdim, int32_t d_state, int32_t ngroups,
                   int32_t io_dtype, const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const void* B,
                   int64_t B_stride, const void* C, int64_t C_stride, const int32_t* seq_idx, const float* dt_bias,
                   const float* A, const float* D, const float* state_in, const void* dy, int64_t dy_stride,
                   const float* dstate_out, void* dx, void* ddt, void* dB, void* dC, float* ddt_bias, float* dA,
                   float* dD, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_dims(batch, seqlen, nheads, headdim, d_state, ngroups, io_dtype);
  if (st) return st;
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch) * seqlen;
  const int64_t wx = static_cast<int64_t>(nheads) * headdim, wb = static_cast<int64_t>(ngroups) * d_state;
  const Rows in[] = {{"x", x, x_stride, wx, 16}, {"dt", dt, dt_stride, nheads, es}, {"B", B, B_stride, wb, 16},
                     {"C", C, C_stride, wb, 16}, {"dy", dy, dy_stride, wx, 16}};
  for (const Rows& r : in) {
    if (!r.p) return fail(MAMBA_ERR_NULL, "%s is NULL", r.name);
    if (r.stride < r.width || r.stride > kMaxStride)
      return fail(MAMBA_ERR_SHAPE, "%s_stride (%lld) must lie in [%lld, 2^24]", r.name, static_cast<long long>(r.stride),
                  static_cast<long long>(r.width));
    if (!aligned(r.p, r.align) || (static_cast<size_t>(r.stride) * es) % r.align != 0)
      return fail(MAMBA_ERR_ALIGN, "%s and its rows must be %zu-byte aligned", r.name, r.align);
  }
  const struct { const char* name; const void* p; size_t align; bool required; } other[] = {
      {"dt_bias", dt_bias, 4, true}, {"A", A, 4, true}, {"D", D, 4, true}, {"seq_idx", seq_idx, 4, false},
      {"state_in", state_in, 16, false}, {"dstate_out", dstate_out, 16, false}, {"dx", dx, 16, true},
      {"ddt", ddt, es, true}, {"dB", dB, 16, true}, {"dC", dC, 16, true}, {"ddt_bias", ddt_bias, 4, true},
      {"dA", dA, 4, true}, {"dD", dD, 4, true}, {"dstate_in", dstate_in, 16, false}};
  for (const auto& o : other) {
    if (o.required && !o.p) return fail(MAMBA_ERR_NULL, "%s is NULL", o.name);
    if (!aligned(o.p, o.align)) return fail(MAMBA_ERR_ALIGN, "%s must be %zu-byte aligned", o.name, o.align);
  }
  const size_t bx = rows * static_cast<size_t>(wx) * es, bb = rows * static_cast<size_t>(wb) * es;
  const size_t bp = static_cast<size_t>(nheads) * 4;
  const size_t bs = static_cast<size_t>(batch) * nheads * headdim * d_state * 4;
  const size_t need = mscan::ssd_bwd_ws_bytes(batch, seqlen, nheads, d_state, ngroups);
  Range ins[11];
  int n = 0;
  for (const Rows& r : in)
    ins[n++] = range(r.name, r.p, ((rows - 1) * static_cast<size_t>(r.stride) + static_cast<size_t>(r.width)) * es);
  ins[n++] = range("seq_idx", seq_idx, rows * 4);
  ins[n++] = range("dt_bias", dt_bias, bp);
  ins[n++] = range("A", A, bp);
  ins[n++] = range("D", D, bp);
  ins[n++] = range("state_in", state_in, bs);
  ins[n++] = range("dstate_out", dstate_out, bs);
  const Range outs[] = {range("dx", dx, bx), range("ddt", ddt, rows * nheads * es), range("dB", dB, bb),
                        range("dC", dC, bb), range("ddt_bias", ddt_bias, bp), range("dA", dA, bp), range("dD", dD, bp),
                        range("dstate_in", dstate_in, bs), range("workspace", workspace, need)};
  if ((st = check_alias(ins, n, outs, 9, nullptr, nullptr, 0))) return st;
  if (!workspace) return fail(MAMBA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are required", need);
  if (workspace_bytes < need)
    return fail(MAMBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", workspace_bytes, need);
  if (!aligned(workspace, 256)) return fail(MAMBA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if ((st = check_device())) return st;
  mscan::SsdBwdCall c{};
  c.batch = batch;
  c.seqlen = seqlen;
  c.nheads = nheads;
  c.d_state = d_state;
  c.ngroups = ngroups;
  c.io_dtype = io_dtype;
  c.x = x;
  c.dt = dt;
  c.B = B;
  c.C = C;
  c.dy = dy;
  c.x_row = x_stride;
  c.dt_row = dt_stride;
  c.b_row = B_stride;
  c.c_row = C_stride;
  c.dy_row = dy_stride;
  c.seq_idx = seq_idx;
  c.dt_bias = dt_bias;
  c.A = A;
  c.D = D;
  c.state_in = state_in;
  c.dstate_out = dstate_out;
  c.dx = dx;
  c.ddt = ddt;
  c.dB = dB;
  c.dC = dC;
  c.ddt_bias = ddt_bias;
  c.dA = dA;
  c.dD = dD;
  c.dstate_in = dstate_in;
  c.workspace = static_cast<char*>(workspace);
  c.stream = static_cast<hipStream_t>(stream);
  const hipError_t err = mscan::launch_ssd_bwd(c);
  if (err != hipSuccess) return fail(MAMBA_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(err));
  count_call();
  return ok();
}

}  // extern "C"
