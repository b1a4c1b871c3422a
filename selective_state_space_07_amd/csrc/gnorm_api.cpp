// C-ABI layer of the group norm (declared in include/mamba_gnorm.h): argument
// validation before any HIP call.
#include "../../include/mamba_gnorm.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "gnorm_internal.h"

namespace {

using namespace mscan::api;

constexpr int64_t kMaxStride = int64_t{1} << 24;

int check_dims(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype) {
  if (rows < 1 || channels < 1 || groups < 1)
    return fail(MAMBA_ERR_SHAPE, "dims must be >= 1 (rows=%lld channels=%d groups=%d)", static_cast<long long>(rows),
                channels, groups);
  // the workgroups of one launch stay far below 2^32 work-items, one to a group at the most
  if (channels > (1 << 20)) return fail(MAMBA_ERR_SHAPE, "channels must be <= 2^20 (got %d)", channels);
  if (channels % groups != 0)
    return fail(MAMBA_ERR_SHAPE, "groups (%d) must divide channels (%d)", groups, channels);
  if (channels / groups > mscan::kGnMaxGroup)
    return fail(MAMBA_ERR_SHAPE, "a group has at most %d channels (got %d)", mscan::kGnMaxGroup, channels / groups);
  if (!below_2_31({rows, groups})) return fail(MAMBA_ERR_SHAPE, "rows * groups must be below 2^31");
  if (io_dtype != MAMBA_F32 && io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_DTYPE, "io_dtype must be MAMBA_F32 (0) or MAMBA_BF16 (1), got %d", io_dtype);
  return MAMBA_OK;
}

int check_rows(const char* name, const void* p, int64_t stride, int32_t channels, size_t es) {
  if (!p) return fail(MAMBA_ERR_NULL, "%s is NULL", name);
  if (stride < channels || stride > kMaxStride)
    return fail(MAMBA_ERR_SHAPE, "%s_stride (%lld) must lie in [channels, 2^24]", name, static_cast<long long>(stride));
  if (!aligned(p, es)) return fail(MAMBA_ERR_ALIGN, "%s must be %zu-byte aligned", name, es);
  return MAMBA_OK;
}

int check_common(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int32_t activation, int32_t gate,
                 float eps, const void* x, int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                 const float* bias) {
  int st = check_dims(rows, channels, groups, io_dtype);
  if (st) return st;
  if (activation < MAMBA_ACT_NONE || activation > MAMBA_ACT_SIGMOID)
    return fail(MAMBA_ERR_SHAPE, "activation must be a MAMBA_ACT_ value (got %d)", activation);
  if (gate < MAMBA_GATE_NONE || gate > MAMBA_GATE_FIRST)
    return fail(MAMBA_ERR_SHAPE, "gate must be a MAMBA_GATE_ value (got %d)", gate);
  if (!(eps >= 0.0f)) return fail(MAMBA_ERR_SHAPE, "eps must be >= 0 (got %g)", static_cast<double>(eps));
  const size_t es = io_size(io_dtype);
  if ((st = check_rows("x", x, x_stride, channels, es))) return st;
  if (gate != MAMBA_GATE_NONE && (st = check_rows("z", z, z_stride, channels, es))) return st;
  if (gate == MAMBA_GATE_NONE && z) return fail(MAMBA_ERR_SHAPE, "z is given but gate is MAMBA_GATE_NONE");
  if (!aligned(weight, 4) || !aligned(bias, 4))
    return fail(MAMBA_ERR_ALIGN, "float32 pointers must be 4-byte aligned");
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

}  // namespace

extern "C" {

int mamba_gnorm_fwd(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int32_t activation,
                    int32_t gate, int32_t center, float eps, const void* x, int64_t x_stride, const void* z,
                    int64_t z_stride, const float* weight, const float* bias, void* y, void* stream) {
  int st = check_common(rows, channels, groups, io_dtype, activation, gate, eps, x, x_stride, z, z_stride, weight, bias);
  if (st) return st;
  const size_t es = io_size(io_dtype);
  if (!y) return fail(MAMBA_ERR_NULL, "y is NULL");
  if (!aligned(y, es)) return fail(MAMBA_ERR_ALIGN, "y must be %zu-byte aligned", es);
  const size_t par = static_cast<size_t>(channels) * 4;
  const Range ins[] = {rows_range("x", x, rows, x_stride, channels, es), rows_range("z", z, rows, z_stride, channels, es),
                       range("weight", weight, par), range("bias", bias, par)};
  const Range outs[] = {rows_range("y", y, rows, channels, channels, es)};
  st = check_alias(ins, 4, outs, 1, nullptr, nullptr, 0);
  if (st) return st;
  if ((st = check_device())) return st;
  mscan::GnCall c{};
  c.rows = rows;
  c.channels = channels;
  c.groups = groups;
  c.io_dtype = io_dtype;
  c.activation = activation;
  c.gate = gate;
  c.center = center;
  c.eps = eps;
  c.x = x;
  c.z = z;
  c.x_row = x_stride;
  c.z_row = z_stride;
  c.weight = weight;
  c.bias = bias;
  c.out = y;
  c.stream = static_cast<hipStream_t>(stream);
  return launched(mscan::launch_gnorm(c));
}

size_t mamba_gnorm_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype,
                                       int32_t want_dweight, int32_t want_dbias) {
  const std::string saved = last_error();
  const int st = check_dims(rows, channels, groups, io_dtype);
  last_error() = saved;
  if (st) return 0;
  return mscan::gn_part_floats(rows, channels, groups, io_dtype, (want_dweight != 0) + (want_dbias != 0)) *
         sizeof(float);
}

int mamba_gnorm_bwd(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int32_t activation,
                    int32_t gate, int32_t center, float eps, const void* x, int64_t x_stride, const void* z,
                    int64_t z_stride, const float* weight, const float* bias, const void* dy, int64_t dy_stride,
                    void* dx, void* dz, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int st = check_common(rows, channels, groups, io_dtype, activation, gate, eps, x, x_stride, z, z_stride, weight, bias);
  if (st) return st;
  const size_t es = io_size(io_dtype);
  if ((st = check_rows("dy", dy, dy_stride, channels, es))) return st;
  if (!dx) return fail(MAMBA_ERR_NULL, "dx is NULL");
  if (gate != MAMBA_GATE_NONE && !dz) return fail(MAMBA_ERR_NULL, "dz is NULL");
  if (gate == MAMBA_GATE_NONE && dz) return fail(MAMBA_ERR_SHAPE, "dz is given but gate is MAMBA_GATE_NONE");
  if (!aligned(dx, es) || !aligned(dz, es)) return fail(MAMBA_ERR_ALIGN, "dx and dz must be %zu-byte aligned", es);
  if (!aligned(dweight, 4) || !aligned(dbias, 4))
    return fail(MAMBA_ERR_ALIGN, "float32 pointers must be 4-byte aligned");
  const size_t par = static_cast<size_t>(channels) * 4;
  const size_t need =
      mscan::gn_part_floats(rows, channels, groups, io_dtype, (dweight != nullptr) + (dbias != nullptr)) * sizeof(float);
  const Range ins[] = {rows_range("x", x, rows, x_stride, channels, es), rows_range("z", z, rows, z_stride, channels, es),
                       rows_range("dy", dy, rows, dy_stride, channels, es), range("weight", weight, par),
                       range("bias", bias, par)};
  const Range outs[] = {rows_range("dx", dx, rows, channels, channels, es),
                        rows_range("dz", dz, rows, channels, channels, es), range("dweight", dweight, par),
                        range("dbias", dbias, par), range("workspace", workspace, need)};
  st = check_alias(ins, 5, outs, 5, nullptr, nullptr, 0);
  if (st) return st;
  if (need) {
    if (!workspace) return fail(MAMBA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are required", need);
    if (workspace_bytes < need)
      return fail(MAMBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", workspace_bytes, need);
    if (!aligned(workspace, 256)) return fail(MAMBA_ERR_ALIGN, "workspace must be 256-byte aligned");
  }
  if ((st = check_device())) return st;
  mscan::GnCall c{};
  c.rows = rows;
  c.channels = channels;
  c.groups = groups;
  c.io_dtype = io_dtype;
  c.activation = activation;
  c.gate = gate;
  c.center = center;
  c.eps = eps;
  c.x = x;
  c.z = z;
  c.dy = dy;
  c.x_row = x_stride;
  c.z_row = z_stride;
  c.dy_row = dy_stride;
  c.weight = weight;
  c.bias = bias;
  c.out = dx;
  c.dz = dz;
  c.dweight = dweight;
  c.dbias = dbias;
  c.part = static_cast<float*>(workspace);
  c.stream = static_cast<hipStream_t>(stream);
  return launched(mscan::launch_gnorm(c));
}

}  // extern "C"
