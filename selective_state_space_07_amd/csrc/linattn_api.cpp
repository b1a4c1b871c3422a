// C-ABI layer of linear attention with a decay for each head (declared in
// include/mamba_linattn.h): argument validation before any HIP call, planning
// and the workspace's layout.
#include "../../include/mamba_linattn.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "linattn_internal.h"

namespace {

using namespace mscan::api;

constexpr int64_t kMaxStride = int64_t{1} << 24;

struct Dims {
  int32_t batch, seqlen, nheads, ngroups, d_k, d_v, io_dtype;
};

int check_dims(const Dims& d) {
  if (d.batch < 1 || d.seqlen < 1 || d.nheads < 1 || d.ngroups < 1)
    return fail(MAMBA_ERR_SHAPE, "dims must be >= 1 (batch=%d seqlen=%d nheads=%d ngroups=%d)", d.batch, d.seqlen,
                d.nheads, d.ngroups);
  if (d.d_k < 8 || d.d_k > 128 || d.d_k % 8 != 0 || d.d_v < 8 || d.d_v > 128 || d.d_v % 8 != 0)
    return fail(MAMBA_ERR_SHAPE, "d_k and d_v must be multiples of 8 in [8, 128] (got %d, %d)", d.d_k, d.d_v);
  if (d.nheads % d.ngroups != 0)
    return fail(MAMBA_ERR_SHAPE, "ngroups (%d) must divide nheads (%d)", d.ngroups, d.nheads);
  // the workgroups of one launch stay below 2^24 (2^32 work-items)
  if (d.nheads > 4096 || static_cast<int64_t>(d.batch) * d.nheads > (int64_t{1} << 20))
    return fail(MAMBA_ERR_SHAPE, "nheads must be <= 4096 and batch * nheads <= 2^20 (got %d, %d)", d.nheads, d.batch);
  if (d.seqlen > (1 << 30) || !below_2_31({d.batch, d.seqlen}))
    return fail(MAMBA_ERR_SHAPE, "seqlen must be <= 2^30 and batch * seqlen < 2^31 (got %d, %d)", d.seqlen, d.batch);
  if (d.io_dtype != MAMBA_F32 && d.io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_DTYPE, "io_dtype must be MAMBA_F32 (0) or MAMBA_BF16 (1), got %d", d.io_dtype);
  return MAMBA_OK;
}

// An io tensor whose rows (b, t) are `stride` elements apart.
struct Rows {
  const char* name;
  const void* p;
  int64_t stride;
  int64_t width;
};

int check_rows(const Rows& r, size_t es, size_t align) {
  if (!r.p) return fail(MAMBA_ERR_NULL, "%s is NULL", r.name);
  if (r.stride < r.width || r.stride > kMaxStride)
    return fail(MAMBA_ERR_SHAPE, "%s_stride (%lld) must lie in [%lld, 2^24]", r.name, static_cast<long long>(r.stride),
                static_cast<long long>(r.width));
  if (!aligned(r.p, align) || (static_cast<size_t>(r.stride) * es) % align != 0)
    return fail(MAMBA_ERR_ALIGN, "%s and its row stride must be %zu-byte aligned", r.name, align);
  return MAMBA_OK;
}

Range rows_range(const Rows& r, size_t rows, size_t es) {
  return range(r.name, r.p, ((rows - 1) * static_cast<size_t>(r.stride) + static_cast<size_t>(r.width)) * es);
}

int check_f32(const char* name, const void* p, bool required, size_t align) {
  if (required && !p) return fail(MAMBA_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, align)) return fail(MAMBA_ERR_ALIGN, "%s must be %zu-byte aligned", name, align);
  return MAMBA_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return MAMBA_OK;
  if (!workspace) return fail(MAMBA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are required", need);
  if (bytes < need) return fail(MAMBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", bytes, need);
  if (!aligned(workspace, 256)) return fail(MAMBA_ERR_ALIGN, "workspace must be 256-byte aligned");
  return MAMBA_OK;
}

mscan::LaPlan plan_fwd(const Dims& d) {
  return mscan::la_plan(d.batch, d.seqlen, d.nheads, d.ngroups, d.d_k, d.d_v, 1);
}
mscan::LaPlan plan_bwd(const Dims& d) {
  return mscan::la_plan(d.batch, d.seqlen, d.nheads, d.ngroups, d.d_k, d.d_v, 3);
}
size_t fwd_floats(const Dims& d) { return mscan::la_ws_floats(plan_fwd(d), d.batch, d.nheads, d.d_k, d.d_v, 1); }
// The backward's workspace: segment states, then dq and dk of every head.
struct BwdWs {
  size_t dq, dk, total;
};
BwdWs bwd_ws(const Dims& d) {
  BwdWs w;
  w.dq = mscan::la_ws_floats(plan_bwd(d), d.batch, d.nheads, d.d_k, d.d_v, 3);
  const size_t part = d.ngroups == d.nheads ? 0 : static_cast<size_t>(d.batch) * d.seqlen * d.nheads * d.d_k;
  w.dk = w.dq + part;
  w.total = w.dk + part;
  return w;
}

bool valid(const Dims& d) {
  const std::string saved = last_error();
  const int st = check_dims(d);
  last_error() = saved;
  return st == MAMBA_OK;
}

int launched(hipError_t err) {
  if (err != hipSuccess) return fail(MAMBA_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(err));
  count_call();
  return ok();
}

}  // namespace

extern "C" {

size_t mamba_linattn_fwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups,
                                         int32_t d_k, int32_t d_v, int32_t io_dtype) {
  const Dims d{batch, seqlen, nheads, ngroups, d_k, d_v, io_dtype};
  return valid(d) ? fwd_floats(d) * sizeof(float) : 0;
}

size_t mamba_linattn_bwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups,
                                         int32_t d_k, int32_t d_v, int32_t io_dtype) {
  const Dims d{batch, seqlen, nheads, ngroups, d_k, d_v, io_dtype};
  return valid(d) ? bwd_ws(d).total * sizeof(float) : 0;
}

int mamba_linattn_fwd(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v,
                      int32_t io_dtype, float scale, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq_idx,
                      const float* log_decay, const float* state_in, void* y, float* state_out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const Dims d{batch, seqlen, nheads, ngroups, d_k, d_v, io_dtype};
  int st = check_dims(d);
  if (st) return st;
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch) * seqlen;
  const int64_t wqk = static_cast<int64_t>(ngroups) * d_k, wv = static_cast<int64_t>(nheads) * d_v;
  const Rows rq{"q", q, q_stride, wqk}, rk{"k", k, k_stride, wqk}, rv{"v", v, v_stride, wv};
  for (const Rows* r : {&rq, &rk, &rv})
    if ((st = check_rows(*r, es, 16))) return st;
  if (!y) return fail(MAMBA_ERR_NULL, "y is NULL");
  if (!aligned(y, 16)) return fail(MAMBA_ERR_ALIGN, "y must be 16-byte aligned");
  if ((st = check_f32("log_decay", log_decay, true, 4))) return st;
  if ((st = check_f32("seq_idx", seq_idx, false, 4))) return st;
  if ((st = check_f32("state_in", state_in, false, 16))) return st;
  if ((st = check_f32("state_out", state_out, false, 16))) return st;
  const size_t need = fwd_floats(d) * sizeof(float);
  const size_t bst = static_cast<size_t>(batch) * nheads * d_v * d_k * 4;
  const Range ins[] = {rows_range(rq, rows, es), rows_range(rk, rows, es), rows_range(rv, rows, es),
                       range("seq_idx", seq_idx, rows * 4), range("log_decay", log_decay, static_cast<size_t>(nheads) * 4),
                       range("state_in", state_in, bst)};
  const Range outs[] = {range("y", y, rows * static_cast<size_t>(wv) * es), range("state_out", state_out, bst),
                        range("workspace", workspace, need)};
  st = check_alias(ins, 6, outs, 3, &ins[5], &outs[1], 1);
  if (st) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if ((st = check_device())) return st;
  mscan::LaCall c{batch, seqlen, nheads, ngroups, io_dtype, seq_idx, log_decay, 1, {},
                  static_cast<float*>(workspace), static_cast<hipStream_t>(stream)};
  c.role[0] = mscan::LaRole{{q, q_stride, true}, {k, k_stride, true}, {v, v_stride, false}, d_k, d_v, y, false,
                            state_in, false, state_out, scale, 1.0f, false, 1, true};
  return launched(mscan::launch_la(c, plan_fwd(d)));
}

int mamba_linattn_bwd(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v,
                      int32_t io_dtype, float scale, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq_idx,
                      const float* log_decay, const float* state_in, const void* dy, int64_t dy_stride,
                      const float* dstate_out, void* dq, void* dk, void* dv, float* dstate_in, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const Dims d{batch, seqlen, nheads, ngroups, d_k, d_v, io_dtype};
  int st = check_dims(d);
  if (st) return st;
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch) * seqlen;
  const int64_t wqk = static_cast<int64_t>(ngroups) * d_k, wv = static_cast<int64_t>(nheads) * d_v;
  const Rows rq{"q", q, q_stride, wqk}, rk{"k", k, k_stride, wqk}, rv{"v", v, v_stride, wv}, rdy{"dy", dy, dy_stride, wv};
  for (const Rows* r : {&rq, &rk, &rv, &rdy})
    if ((st = check_rows(*r, es, 16))) return st;
  const struct { const void* p; const char* n; } io_outs[] = {{dq, "dq"}, {dk, "dk"}, {dv, "dv"}};
  for (const auto& o : io_outs) {
    if (!o.p) return fail(MAMBA_ERR_NULL, "%s is NULL", o.n);
    if (!aligned(o.p, 16)) return fail(MAMBA_ERR_ALIGN, "%s must be 16-byte aligned", o.n);
  }
  if ((st = check_f32("log_decay", log_decay, true, 4))) return st;
  if ((st = check_f32("seq_idx", seq_idx, false, 4))) return st;
  if ((st = check_f32("state_in", state_in, false, 16))) return st;
  if ((st = check_f32("dstate_out", dstate_out, false, 16))) return st;
  if ((st = check_f32("dstate_in", dstate_in, false, 16))) return st;
  const BwdWs w = bwd_ws(d);
  const size_t need = w.total * sizeof(float);
  const size_t bst = static_cast<size_t>(batch) * nheads * d_v * d_k * 4;
  const size_t bqk = rows * static_cast<size_t>(wqk) * es;
  const Range ins[] = {rows_range(rq, rows, es), rows_range(rk, rows, es), rows_range(rv, rows, es),
                       rows_range(rdy, rows, es), range("seq_idx", seq_idx, rows * 4),
                       range("log_decay", log_decay, static_cast<size_t>(nheads) * 4), range("state_in", state_in, bst),
                       range("dstate_out", dstate_out, bst)};
  const Range outs[] = {range("dq", dq, bqk), range("dk", dk, bqk), range("dv", dv, rows * static_cast<size_t>(wv) * es),
                        range("dstate_in", dstate_in, bst), range("workspace", workspace, need)};
  st = check_alias(ins, 8, outs, 5, nullptr, nullptr, 0);
  if (st) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need))) return st;
  if ((st = check_device())) return st;
  float* ws = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool shared = ngroups != nheads;
  void* dq_to = shared ? ws + w.dq : dq;
  void* dk_to = shared ? ws + w.dk : dk;
  mscan::LaCall c{batch, seqlen, nheads, ngroups, io_dtype, seq_idx, log_decay, 3, {}, ws, s};
  const mscan::LaOperand oq{q, q_stride, true}, ok_{k, k_stride, true}, ov{v, v_stride, false}, ody{dy, dy_stride, false};
  c.role[0] = mscan::LaRole{ody, ov, ok_, d_v, d_k, dq_to, shared, state_in, true, nullptr, scale, 1.0f, false, 1, false};
  c.role[1] = mscan::LaRole{ov, ody, oq, d_v, d_k, dk_to, shared, dstate_out, true, nullptr, 1.0f, scale, true, 0, false};
  c.role[2] = mscan::LaRole{ok_, oq, ody, d_k, d_v, dv, false, dstate_out, false, dstate_in, 1.0f, scale, true, 0, true};
  hipError_t err = mscan::launch_la(c, plan_bwd(d));
  if (err == hipSuccess && shared)
    err = mscan::launch_la_head_sum(static_cast<int64_t>(rows), nheads, ngroups, d_k, io_dtype, ws + w.dq, dq, s);
  if (err == hipSuccess && shared)
    err = mscan::launch_la_head_sum(static_cast<int64_t>(rows), nheads, ngroups, d_k, io_dtype, ws + w.dk, dk, s);
  return launched(err);
}

int mamba_linattn_step(int32_t batch, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v, int32_t io_dtype,
                       float scale, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const float* log_decay, const float* state_in, void* y, float* state_out,
                       void* stream) {
  int st = check_dims(Dims{batch, 1, nheads, ngroups, d_k, d_v, io_dtype});
  if (st) return st;
  if (!below_2_31({batch, nheads, d_v})) return fail(MAMBA_ERR_SHAPE, "batch * nheads * d_v must be below 2^31");
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch);
  const int64_t wqk = static_cast<int64_t>(ngroups) * d_k, wv = static_cast<int64_t>(nheads) * d_v;
  const Rows rq{"q", q, q_stride, wqk}, rk{"k", k, k_stride, wqk}, rv{"v", v, v_stride, wv};
  for (const Rows* r : {&rq, &rk, &rv})
    if ((st = check_rows(*r, es, es))) return st;
  if (!y) return fail(MAMBA_ERR_NULL, "y is NULL");
  if (!aligned(y, es)) return fail(MAMBA_ERR_ALIGN, "y must be %zu-byte aligned", es);
  if ((st = check_f32("log_decay", log_decay, true, 4))) return st;
  if ((st = check_f32("state_in", state_in, true, 16))) return st;
  if ((st = check_f32("state_out", state_out, true, 16))) return st;
  const size_t bst = static_cast<size_t>(batch) * nheads * d_v * d_k * 4;
  const Range ins[] = {rows_range(rq, rows, es), rows_range(rk, rows, es), rows_range(rv, rows, es),
                       range("log_decay", log_decay, static_cast<size_t>(nheads) * 4), range("state_in", state_in, bst)};
  const Range outs[] = {range("y", y, rows * static_cast<size_t>(wv) * es), range("state_out", state_out, bst)};
  st = check_alias(ins, 5, outs, 2, &ins[4], &outs[1], 1);
  if (st) return st;
  if ((st = check_device())) return st;
  const mscan::LaStepCall c{batch, nheads, ngroups, d_k, d_v, io_dtype, scale, q, k, v, q_stride, k_stride, v_stride,
                            log_decay, state_in, y, state_out, static_cast<hipStream_t>(stream)};
  return launched(mscan::launch_la_step(c));
}

}  // extern "C"
