// C-ABI layer of the RMS norm with the residual's addition (declared in
// include/mamba_rmsnorm.h): argument validation before any HIP call.
#include "../../include/mamba_rmsnorm.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "rmsnorm_internal.h"

namespace {

using namespace mscan::api;

constexpr int64_t kMaxStride = int64_t{1} << 24;

int check_dims(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype) {
  if (rows < 1 || channels < 1)
    return fail(MAMBA_ERR_SHAPE, "dims must be >= 1 (rows=%lld channels=%d)", static_cast<long long>(rows), channels);
  if (channels > mscan::kRnMaxChannels)
    return fail(MAMBA_ERR_SHAPE, "channels must be <= %d (got %d)", mscan::kRnMaxChannels, channels);
  if (rows >= (int64_t{1} << 31)) return fail(MAMBA_ERR_SHAPE, "rows must be below 2^31");
  if (io_dtype != MAMBA_F32 && io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_DTYPE, "io_dtype must be MAMBA_F32 (0) or MAMBA_BF16 (1), got %d", io_dtype);
  if (residual_dtype != MAMBA_F32 && (residual_dtype != MAMBA_BF16 || io_dtype != MAMBA_BF16))
    return fail(MAMBA_ERR_DTYPE, "residual_dtype must be MAMBA_F32, or MAMBA_BF16 like io_dtype, got %d", residual_dtype);
  return MAMBA_OK;
}

int check_eps(float eps) {
  return eps >= 0.0f ? MAMBA_OK : fail(MAMBA_ERR_SHAPE, "eps must be >= 0 (got %g)", static_cast<double>(eps));
}

int check_rows(const char* name, const void* p, int64_t stride, int32_t channels, size_t es, size_t align) {
  if (!p) return fail(MAMBA_ERR_NULL, "%s is NULL", name);
  if (stride < channels || stride > kMaxStride)
    return fail(MAMBA_ERR_SHAPE, "%s_stride (%lld) must lie in [channels, 2^24]", name, static_cast<long long>(stride));
  if (!aligned(p, align) || (static_cast<size_t>(stride) * es) % align != 0)
    return fail(MAMBA_ERR_ALIGN, "%s and its rows must be %zu-byte aligned", name, align);
  return MAMBA_OK;
}

Range rows_range(const char* name, const void* p, int64_t rows, int64_t stride, int32_t channels, size_t es) {
  return range(name, p, (static_cast<size_t>(rows - 1) * static_cast<size_t>(stride) + channels) * es);
}

int launched(hipError_t err) {
  if (err != hipSuccess) return fail(MAMBA_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(err));
  count_call();
  return ok();
}

int run_fwd(mscan::RnCall& c, bool fp8) {
  int st = check_dims(c.rows, c.channels, c.io_dtype, c.residual_dtype);
  if (st) return st;
  if ((st = check_eps(c.eps))) return st;
  if (c.block != 0 && c.block != 128) return fail(MAMBA_ERR_SHAPE, "block must be 0 or 128 (got %d)", c.block);
  if (fp8 && c.channels % 16 != 0)
    return fail(MAMBA_ERR_SHAPE, "channels must be a multiple of 16 for 8-bit outputs (got %d)", c.channels);
  const size_t es = io_size(c.io_dtype), rs = io_size(c.residual_dtype), os = fp8 ? 1 : es;
  if ((st = check_rows("x", c.x, c.x_row, c.channels, es, fp8 ? 16 : es))) return st;
  if (c.residual && (st = check_rows("residual", c.residual, c.residual_row, c.channels, rs, fp8 ? 16 : rs))) return st;
  if (!c.y) return fail(MAMBA_ERR_NULL, "y is NULL");
  if (fp8 && !c.scales) return fail(MAMBA_ERR_NULL, "scales is NULL");
  if (!aligned(c.y, fp8 ? 16 : os) || !aligned(c.h_out, fp8 ? 16 : rs))
    return fail(MAMBA_ERR_ALIGN, "y and h must be %s aligned", fp8 ? "16-byte" : "element");
  if (!aligned(c.weight, 4) || !aligned(c.scales, 4))
    return fail(MAMBA_ERR_ALIGN, "float32 pointers must be 4-byte aligned");
  const size_t nscales = static_cast<size_t>(c.rows) * (c.block ? (c.channels + c.block - 1) / c.block : 1);
  const Range ins[] = {rows_range("x", c.x, c.rows, c.x_row, c.channels, es),
                       rows_range("residual", c.residual, c.rows, c.residual_row, c.channels, rs),
                       range("weight", c.weight, static_cast<size_t>(c.channels) * 4)};
  const Range outs[] = {rows_range("y", c.y, c.rows, c.channels, c.channels, os),
                        rows_range("h", c.h_out, c.rows, c.channels, c.channels, rs),
                        range("scales", c.scales, nscales * 4)};
  if ((st = check_alias(ins, 3, outs, 3, &ins[1], &outs[1], 1))) return st;
  if ((st = check_device())) return st;
  return launched(mscan::launch_rmsnorm(c));
}

mscan::RnCall fwd_call(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                       const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                       const float* weight, void* y, void* h, void* stream) {
  mscan::RnCall c{};
  c.rows = rows;
  c.channels = channels;
  c.io_dtype = io_dtype;
  c.residual_dtype = residual_dtype;
  c.eps = eps;
  c.x = x;
  c.x_row = x_stride;
  c.residual = residual;
  c.residual_row = residual_stride;
  c.weight = weight;
  c.y = y;
  c.h_out = h;
  c.stream = static_cast<hipStream_t>(stream);
  return c;
}

}  // namespace

extern "C" {

int mamba_rmsnorm_fwd(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                      const float* weight, void* y, void* h, void* stream) {
  mscan::RnCall c = fwd_call(rows, channels, io_dtype, residual_dtype, eps, x, x_stride, residual, residual_stride,
                             weight, y, h, stream);
  return run_fwd(c, false);
}

int mamba_rmsnorm_fp8(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      int32_t block, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                      const float* weight, void* y8, float* scales, void* h, void* stream) {
  mscan::RnCall c = fwd_call(rows, channels, io_dtype, residual_dtype, eps, x, x_stride, residual, residual_stride,
                             weight, y8, h, stream);
  c.block = block;
  c.scales = scales;
  return run_fwd(c, true);
}

size_t mamba_rmsnorm_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype,
                                         int32_t want_dweight) {
  const std::string saved = last_error();
  const int st = check_dims(rows, channels, io_dtype, residual_dtype);
  last_error() = saved;
  return st || !want_dweight ? 0 : mscan::rn_part_floats(rows, channels, io_dtype) * sizeof(float);
}

int mamba_rmsnorm_bwd(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      const void* h, int64_t h_stride, const float* weight, const void* dy, int64_t dy_stride,
                      const void* dh, int64_t dh_stride, void* dx, void* dresidual, float* dweight, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int st = check_dims(rows, channels, io_dtype, residual_dtype);
  if (st) return st;
  if ((st = check_eps(eps))) return st;
  const size_t es = io_size(io_dtype), rs = io_size(residual_dtype), par = static_cast<size_t>(channels) * 4;
  if ((st = check_rows("h", h, h_stride, channels, rs, rs))) return st;
  if ((st = check_rows("dy", dy, dy_stride, channels, es, es))) return st;
  if (dh && (st = check_rows("dh", dh, dh_stride, channels, rs, rs))) return st;
  if (!dx && !dresidual) return fail(MAMBA_ERR_NULL, "dx and dresidual are NULL");
  if (!aligned(dx, es) || !aligned(dresidual, rs))
    return fail(MAMBA_ERR_ALIGN, "dx and dresidual must be element aligned");
  if (!aligned(weight, 4) || !aligned(dweight, 4))
    return fail(MAMBA_ERR_ALIGN, "float32 pointers must be 4-byte aligned");
  const size_t need = dweight ? mscan::rn_part_floats(rows, channels, io_dtype) * sizeof(float) : 0;
  const Range ins[] = {rows_range("h", h, rows, h_stride, channels, rs), rows_range("dy", dy, rows, dy_stride, channels, es),
                       rows_range("dh", dh, rows, dh_stride, channels, rs), range("weight", weight, par)};
  const Range outs[] = {rows_range("dx", dx, rows, channels, channels, es),
                        rows_range("dresidual", dresidual, rows, channels, channels, rs), range("dweight", dweight, par),
                        range("workspace", workspace, need)};
  if ((st = check_alias(ins, 4, outs, 4, &ins[2], &outs[1], 1))) return st;
  if (need) {
    if (!workspace) return fail(MAMBA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are required", need);
    if (workspace_bytes < need)
      return fail(MAMBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", workspace_bytes, need);
    if (!aligned(workspace, 256)) return fail(MAMBA_ERR_ALIGN, "workspace must be 256-byte aligned");
  }
  if ((st = check_device())) return st;
  mscan::RnCall c{};
  c.rows = rows;
  c.channels = channels;
  c.io_dtype = io_dtype;
  c.residual_dtype = residual_dtype;
  c.eps = eps;
  c.h = h;
  c.h_row = h_stride;
  c.weight = weight;
  c.dy = dy;
  c.dy_row = dy_stride;
  c.dh = dh;
  c.dh_row = dh_stride;
  c.dx = dx;
  c.dresidual = dresidual;
  c.dweight = dweight;
  c.part = static_cast<float*>(workspace);
  c.stream = static_cast<hipStream_t>(stream);
  return launched(mscan::launch_rmsnorm(c));
}

}  // extern "C"
