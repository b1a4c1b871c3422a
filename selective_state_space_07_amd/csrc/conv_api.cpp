// C-ABI layer of the short causal convolution (declared in
// include/mamba_conv.h): argument validation before any HIP call.
#include "../../include/mamba_conv.h"

#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "conv_internal.h"

namespace {

using namespace mscan::api;

constexpr int64_t kMaxStride = int64_t{1} << 24;
static_assert(MAMBA_CONV_MAX_PARTS == mscan::kConvMaxParts, "one limit");

int check_dims(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype) {
  if (batch < 1 || seqlen < 1 || channels < 1)
    return fail(MAMBA_ERR_SHAPE, "dims must be >= 1 (batch=%d seqlen=%d channels=%d)", batch, seqlen, channels);
  if (taps < 2 || taps > 4) return fail(MAMBA_ERR_SHAPE, "taps must be 2, 3 or 4 (got %d)", taps);
  if (channels > (1 << 20) || batch > (1 << 24))
    return fail(MAMBA_ERR_SHAPE, "channels must be <= 2^20 and batch <= 2^24 (got %d, %d)", channels, batch);
  // (a run's end, and the tokens fetched ahead of it, are int32 numbers)
  if (!below_2_31({2, batch, seqlen})) return fail(MAMBA_ERR_SHAPE, "batch * seqlen must be below 2^30");
  if (io_dtype != MAMBA_F32 && io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_DTYPE, "io_dtype must be MAMBA_F32 (0) or MAMBA_BF16 (1), got %d", io_dtype);
  return MAMBA_OK;
}

int check_rows(const char* name, const void* p, int64_t stride, int32_t width, size_t es) {
  if (!p) return fail(MAMBA_ERR_NULL, "%s is NULL", name);
  if (stride < width || stride > kMaxStride)
    return fail(MAMBA_ERR_SHAPE, "%s_stride (%lld) must lie in [%d, 2^24]", name, static_cast<long long>(stride), width);
  if (!aligned(p, es)) return fail(MAMBA_ERR_ALIGN, "%s must be %zu-byte aligned", name, es);
  return MAMBA_OK;
}

Range rows_range(const char* name, const void* p, size_t rows, int64_t stride, int32_t width, size_t es) {
  return range(name, p, ((rows - 1) * static_cast<size_t>(stride) + static_cast<size_t>(width)) * es);
}

// The call's sizes, x, parameters and parts (`strides` NULL: contiguous).
int fill(mscan::ConvCall& c, const char* part_name, int32_t parts, const int32_t* part_channels, void* const* part,
         const int64_t* strides) {
  int st = check_dims(c.batch, c.seqlen, c.channels, c.taps, c.io_dtype);
  if (st) return st;
  if (c.activation != MAMBA_ACT_NONE && c.activation != MAMBA_ACT_SILU)
    return fail(MAMBA_ERR_SHAPE, "activation must be MAMBA_ACT_NONE or MAMBA_ACT_SILU (got %d)", c.activation);
  const size_t es = io_size(c.io_dtype);
  if ((st = check_rows("x", c.x, c.x_row, c.channels, es))) return st;
  if (!c.weight) return fail(MAMBA_ERR_NULL, "weight is NULL");
  for (const void* p : {static_cast<const void*>(c.weight), static_cast<const void*>(c.bias),
                        static_cast<const void*>(c.state_in), static_cast<const void*>(c.seq_idx)})
    if (!aligned(p, 4)) return fail(MAMBA_ERR_ALIGN, "float32 and int32 pointers must be 4-byte aligned");
  if (parts < 1 || parts > MAMBA_CONV_MAX_PARTS)
    return fail(MAMBA_ERR_SHAPE, "parts must lie in [1, %d] (got %d)", MAMBA_CONV_MAX_PARTS, parts);
  if (!part_channels || !part) return fail(MAMBA_ERR_NULL, "part_channels or %s is NULL", part_name);
  c.parts = parts;
  int64_t sum = 0;
  for (int i = 0; i < parts; ++i) {
    if (part_channels[i] < 1 || part_channels[i] > c.channels)
      return fail(MAMBA_ERR_SHAPE, "part_channels[%d] (%d) must lie in [1, channels]", i, part_channels[i]);
    sum += part_channels[i];
    c.part_channels[i] = part_channels[i];
    c.part[i] = part[i];
    c.part_row[i] = strides ? strides[i] : part_channels[i];
    if ((st = check_rows(part_name, part[i], c.part_row[i], part_channels[i], es))) return st;
  }
  if (sum != c.channels)
    return fail(MAMBA_ERR_SHAPE, "part_channels add up to %lld, not to channels (%d)", static_cast<long long>(sum),
                c.channels);
  return MAMBA_OK;
}

int launched(hipError_t err) {
  if (err != hipSuccess) return fail(MAMBA_ERR_DEVICE, "kernel launch failed: %s", hipGetErrorString(err));
  count_call();
  return ok();
}

size_t state_bytes(const mscan::ConvCall& c) {
  return static_cast<size_t>(c.batch) * c.channels * (c.taps - 1) * 4;
}

}  // namespace

extern "C" {

int mamba_conv_fwd(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype,
                   int32_t activation, const void* x, int64_t x_stride, const int32_t* seq_idx, const float* weight,
                   const float* bias, const float* state_in, int32_t parts, const int32_t* part_channels,
                   void* const* y, float* state_out, void* stream) {
  mscan::ConvCall c{};
  c.batch = batch;
  c.seqlen = seqlen;
  c.channels = channels;
  c.taps = taps;
  c.io_dtype = io_dtype;
  c.activation = activation;
  c.x = x;
  c.x_row = x_stride;
  c.seq_idx = seq_idx;
  c.weight = weight;
  c.bias = bias;
  c.state_in = state_in;
  c.state_out = state_out;
  c.stream = static_cast<hipStream_t>(stream);
  int st = fill(c, "y", parts, part_channels, y, nullptr);
  if (st) return st;
  if (!aligned(state_out, 4)) return fail(MAMBA_ERR_ALIGN, "state_out must be 4-byte aligned");
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch) * seqlen, par = static_cast<size_t>(channels) * 4;
  const Range ins[] = {rows_range("x", x, rows, x_stride, channels, es), range("seq_idx", seq_idx, rows * 4),
                       range("weight", weight, par * taps), range("bias", bias, par),
                       range("state_in", state_in, state_bytes(c))};
  Range outs[MAMBA_CONV_MAX_PARTS + 1];
  for (int i = 0; i < parts; ++i) outs[i] = rows_range("y", y[i], rows, part_channels[i], part_channels[i], es);
  outs[parts] = range("state_out", state_out, state_bytes(c));
  if ((st = check_alias(ins, 5, outs, parts + 1, nullptr, nullptr, 0))) return st;
  if ((st = check_device())) return st;
  return launched(mscan::launch_conv(c));
}

size_t mamba_conv_bwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype) {
  const std::string saved = last_error();
  const int st = check_dims(batch, seqlen, channels, taps, io_dtype);
  last_error() = saved;
  return st ? 0 : mscan::conv_part_floats(batch, seqlen, channels, taps) * sizeof(float);
}

int mamba_conv_bwd(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype,
                   int32_t activation, const void* x, int64_t x_stride, const int32_t* seq_idx, const float* weight,
                   const float* bias, const float* state_in, int32_t parts, const int32_t* part_channels,
                   const void* const* dy, const int64_t* dy_stride, const float* dstate_out, void* dx, float* dweight,
                   float* dbias, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  mscan::ConvCall c{};
  c.batch = batch;
  c.seqlen = seqlen;
  c.channels = channels;
  c.taps = taps;
  c.io_dtype = io_dtype;
  c.activation = activation;
  c.x = x;
  c.x_row = x_stride;
  c.seq_idx = seq_idx;
  c.weight = weight;
  c.bias = bias;
  c.state_in = state_in;
  c.dstate_out = dstate_out;
  c.dx = dx;
  c.dweight = dweight;
  c.dbias = dbias;
  c.dstate_in = dstate_in;
  c.sums = static_cast<float*>(workspace);
  c.stream = static_cast<hipStream_t>(stream);
  int st = check_dims(batch, seqlen, channels, taps, io_dtype);
  if (st) return st;
  if (!dy_stride) return fail(MAMBA_ERR_NULL, "dy_stride is NULL");
  st = fill(c, "dy", parts, part_channels, const_cast<void* const*>(dy), dy_stride);
  if (st) return st;
  if (!dx) return fail(MAMBA_ERR_NULL, "dx is NULL");
  if (!dweight) return fail(MAMBA_ERR_NULL, "dweight is NULL");
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch) * seqlen, par = static_cast<size_t>(channels) * 4;
  if (!aligned(dx, es)) return fail(MAMBA_ERR_ALIGN, "dx must be %zu-byte aligned", es);
  for (const void* p : {static_cast<const void*>(dstate_out), static_cast<const void*>(dweight),
                        static_cast<const void*>(dbias), static_cast<const void*>(dstate_in)})
    if (!aligned(p, 4)) return fail(MAMBA_ERR_ALIGN, "float32 pointers must be 4-byte aligned");
  const size_t need = mscan::conv_part_floats(batch, seqlen, channels, taps) * sizeof(float);
  Range ins[6 + MAMBA_CONV_MAX_PARTS] = {
      rows_range("x", x, rows, x_stride, channels, es), range("seq_idx", seq_idx, rows * 4),
      range("weight", weight, par * taps), range("bias", bias, par), range("state_in", state_in, state_bytes(c)),
      range("dstate_out", dstate_out, state_bytes(c))};
  for (int i = 0; i < parts; ++i) ins[6 + i] = rows_range("dy", dy[i], rows, dy_stride[i], part_channels[i], es);
  const Range outs[] = {rows_range("dx", dx, rows, channels, channels, es), range("dweight", dweight, par * taps),
                        range("dbias", dbias, par), range("dstate_in", dstate_in, state_bytes(c)),
                        range("workspace", workspace, need)};
  if ((st = check_alias(ins, 6 + parts, outs, 5, nullptr, nullptr, 0))) return st;
  if (!workspace) return fail(MAMBA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are required", need);
  if (workspace_bytes < need)
    return fail(MAMBA_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", workspace_bytes, need);
  if (!aligned(workspace, 256)) return fail(MAMBA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if ((st = check_device())) return st;
  return launched(mscan::launch_conv(c));
}

int mamba_conv_step(int32_t batch, int32_t channels, int32_t taps, int32_t io_dtype, int32_t activation, const void* x,
                    int64_t x_stride, const float* weight, const float* bias, const float* state_in, int32_t parts,
                    const int32_t* part_channels, void* const* y, float* state_out, void* stream) {
  mscan::ConvCall c{};
  c.batch = batch;
  c.seqlen = 1;
  c.channels = channels;
  c.taps = taps;
  c.io_dtype = io_dtype;
  c.activation = activation;
  c.x = x;
  c.x_row = x_stride;
  c.weight = weight;
  c.bias = bias;
  c.state_in = state_in;
  c.state_out = state_out;
  c.stream = static_cast<hipStream_t>(stream);
  int st = fill(c, "y", parts, part_channels, y, nullptr);
  if (st) return st;
  if (!state_in) return fail(MAMBA_ERR_NULL, "state_in is NULL");
  if (!state_out) return fail(MAMBA_ERR_NULL, "state_out is NULL");
  if (!aligned(state_out, 4)) return fail(MAMBA_ERR_ALIGN, "state_out must be 4-byte aligned");
  const size_t es = io_size(io_dtype), rows = static_cast<size_t>(batch), par = static_cast<size_t>(channels) * 4;
  const Range ins[] = {rows_range("x", x, rows, x_stride, channels, es), range("weight", weight, par * taps),
                       range("bias", bias, par), range("state_in", state_in, state_bytes(c))};
  Range outs[MAMBA_CONV_MAX_PARTS + 1];
  for (int i = 0; i < parts; ++i) outs[i] = rows_range("y", y[i], rows, part_channels[i], part_channels[i], es);
  outs[parts] = range("state_out", state_out, state_bytes(c));
  const Range pin[] = {ins[3]}, pout[] = {outs[parts]};
  if ((st = check_alias(ins, 4, outs, parts + 1, pin, pout, 1))) return st;
  if ((st = check_device())) return st;
  return launched(mscan::launch_conv_step(c));
}

}  // extern "C"
