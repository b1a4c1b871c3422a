// Group norm over the channels of a row (token), channels last, with an
// activation and a gate, and its gradients.
//
// Per row and group of gs channels, with a = activation(z) for a gate:
//   u  = x a (gate first) or x;   mu = mean(u) (0 without centering)
//   xh = (u - mu) / sqrt(mean((u - mu)^2) + eps);   n = xh w + b
//   y  = n a (gate after), n (gate first) or activation(n) (no gate).
// Gradients, with dn = dy a, dy or dy activation'(n) and dxh = dn w:
//   dw = sum over rows of dn xh,  db = sum over rows of dn,
//   du = (dxh - mean(dxh) - xh mean(dxh xh)) / sqrt(...)  (no mean(dxh) without centering),
//   dx = du a (gate first) or du;  dz = du x act'(z) (first) or dy n act'(z) (after).
// The statistics are taken again in the backward: the group is in registers
// anyway, and nothing of the forward has to be kept.
//
// All tensors are read and written once, so both directions are bound by
// memory traffic. A group is held in registers by 1 to 64 lanes of one wave
// (the power of two that covers it with 16-byte pieces, up to 4 pieces a
// lane), or by a whole workgroup of 256 to 1024 threads; the mean is taken
// first and the squares of what is left of it, in float32. A wave takes
// several neighbouring groups of a row, and several rows, where groups are
// small; it keeps its channels from row to row, so that the sums over rows
// stay in registers and leave as one partial sum per workgroup, which a second
// kernel adds in a fixed order.
#include "gnorm_internal.h"
#include "mfma_frag.h"
#include "scan_device.h"

namespace mscan {

namespace {

constexpr int kWaves = 4;            // waves per workgroup where a wave holds whole groups
constexpr int kGateNone = 0, kGateAfter = 1, kGateFirst = 2;
constexpr int kActNone = 0, kActSilu = 1;  // 2: sigmoid

struct GnArgs {
  int64_t rows, x_row, z_row, dy_row;
  int32_t channels, gs, ln, ln_log, gp, tiles, nblk;  // lanes of a group, groups of a wave's tile, tiles of a row
  int32_t activation, gate, center;
  float eps;
  const void *x, *z, *dy;
  const float *weight, *bias;
  void *out, *dz;
  float *pw, *pb;  // partial sums [nblk][channels], or NULL
};

// A lane's piece of a row: V io elements in one load.
template <int IO, int V>
struct Vec {
  u4 v;
};
template <int IO>
struct Vec<IO, 1> {
  typename Io<IO>::T v;
};
template <int IO, int V>
__device__ __forceinline__ void unpack(const Vec<IO, V>& p, float (&o)[V]) {
  if constexpr (V == 1) {
    o[0] = Io<IO>::cvt(p.v);
  } else if constexpr (IO == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t e = p.v[i];
      o[2 * i] = __uint_as_float(e << 16);
      o[2 * i + 1] = __uint_as_float(e & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t e = p.v[i];
      o[i] = __uint_as_float(e);
    }
  }
}
template <int IO, int V>
__device__ __forceinline__ void put(typename Io<IO>::T* p, const float (&o)[V]) {
  if constexpr (V == 1) {
    Io<IO>::store(p, o[0]);
  } else if constexpr (IO == 1) {
    const bf8 v = {static_cast<__bf16>(o[0]), static_cast<__bf16>(o[1]), static_cast<__bf16>(o[2]),
                   static_cast<__bf16>(o[3]), static_cast<__bf16>(o[4]), static_cast<__bf16>(o[5]),
                   static_cast<__bf16>(o[6]), static_cast<__bf16>(o[7])};
    *reinterpret_cast<u4*>(p) = __builtin_bit_cast(u4, v);
  } else {
    *reinterpret_cast<f4*>(p) = f4{o[0], o[1], o[2], o[3]};
  }
}
template <int IO, int V>
__device__ __forceinline__ Vec<IO, V> fetch(const void* base, int64_t at, bool ok) {
  Vec<IO, V> r{};
  if (ok) r = *reinterpret_cast<const Vec<IO, V>*>(static_cast<const typename Io<IO>::T*>(base) + at);
  return r;
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true);
  return v + __builtin_bit_cast(float, o);
}

// The sum over the 1 to 64 lanes of a group, in all of them (ln is uniform).
// Each step adds a mirrored or exchanged partner, so all lanes hold the same
// bits.
__device__ __forceinline__ float lanes_sum(float v, int ln) {
  if (ln > 1) v = dpp_add<0xB1>(v);   // quad_perm 1,0,3,2
  if (ln > 2) v = dpp_add<0x4E>(v);   // quad_perm 2,3,0,1
  if (ln > 4) v = dpp_add<0x141>(v);  // the other quad of 8
  if (ln > 8) v = dpp_add<0x140>(v);  // the other 8 of a row of 16
  if (ln > 16) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (ln > 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// The same over a whole workgroup; `red` holds one float per wave.
__device__ __forceinline__ float wide_sum(float v, float* red) {
  v = lanes_sum(v, 64);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  __syncthreads();  // the last sum's readers are done
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < waves; ++w) v += red[w];
  return v;
}

// sigmoid(z) and 1 - sigmoid(z), the latter without cancellation. The exponent
// is capped at 100, where 1 + e rounds to e: e sigmoid(z) stays 1, not inf * 0.
struct Sig {
  float s, c;
};
__device__ __forceinline__ Sig sigmoid(float z) {
  float t = -z * kLog2e;
  t = t > 100.0f ? 100.0f : t;
  const float e = exp2_hw(t), s = rcp_hw(1.0f + e);
  return Sig{s, e * s};
}
__device__ __forceinline__ float act(int kind, float z) {
  if (kind == kActNone) return z;
  const float s = sigmoid(z).s;
  return kind == kActSilu ? z * s : s;
}
// activation and its derivative
__device__ __forceinline__ float act_grad(int kind, float z, float& a) {
  if (kind == kActNone) {
    a = z;
    return 1.0f;
  }
  const Sig g = sigmoid(z);
  a = kind == kActSilu ? z * g.s : g.s;
  return kind == kActSilu ? g.s * fmaf(z, g.c, 1.0f) : g.s * g.c;
}

// V elements a piece, K pieces a lane. WIDE: one group of one row per workgroup.
template <int IO, int V, int K, bool WIDE, bool BWD>
__global__ __launch_bounds__(WIDE ? 1024 : 64 * kWaves) void gnorm_kernel(const GnArgs a) {
  using T = typename Io<IO>::T;
  __shared__ float red[WIDE ? 16 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x % a.tiles, blk = blockIdx.x / a.tiles;
  const int in = WIDE ? tid : lane & (a.ln - 1);              // lane within its group
  const int slot = WIDE ? 0 : lane >> a.ln_log;               // which of the wave's groups
  const int sub = WIDE ? 0 : slot / a.gp;                     // which of the wave's rows
  const int rp = WIDE ? 1 : 64 / (a.ln * a.gp);               // rows of a wave
  const int ch0 = (tile * a.gp + (slot - sub * a.gp)) * a.gs;  // the group's first channel
  const int lanes = WIDE ? static_cast<int>(blockDim.x) : a.ln;
  const float inv = 1.0f / static_cast<float>(a.gs);
  auto sum = [&](float v) { return WIDE ? wide_sum(v, red) : lanes_sum(v, a.ln); };

  int ch[K];
  bool in_group[K];
  float w[K][V], b[K][V], sw[BWD ? K : 1][V], sb[BWD ? K : 1][V];
#pragma unroll
  for (int p = 0; p < K; ++p) {
    const int e = (p * lanes + in) * V;
    in_group[p] = e < a.gs;
    ch[p] = ch0 + e;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[p][i] = in_group[p] && a.weight ? a.weight[ch[p] + i] : 1.0f;
      b[p][i] = in_group[p] && a.bias ? a.bias[ch[p] + i] : 0.0f;
      if (BWD) sw[p][i] = sb[p][i] = 0.0f;
    }
  }

  const int64_t per = WIDE ? 1 : static_cast<int64_t>(kWaves) * rp;  // rows of a workgroup
  int64_t row0 = blk * per + (WIDE ? 0 : static_cast<int64_t>(wave) * rp);  // uniform in the wave
  Vec<IO, V> rx[K], rz[K], rd[BWD ? K : 1];
  auto load = [&](int64_t r0) {
    const int64_t row = r0 + sub;
#pragma unroll
    for (int p = 0; p < K; ++p) {
      const bool ok = in_group[p] && row < a.rows;
      rx[p] = fetch<IO, V>(a.x, row * a.x_row + ch[p], ok);
      if (a.gate != kGateNone) rz[p] = fetch<IO, V>(a.z, row * a.z_row + ch[p], ok);
      if (BWD) rd[p] = fetch<IO, V>(a.dy, row * a.dy_row + ch[p], ok);
    }
  };
  if (row0 < a.rows) load(row0);
  for (; row0 < a.rows; row0 += per * a.nblk) {
    const int64_t row = row0 + sub;
    float x[K][V], z[K][V], d[BWD ? K : 1][V];
#pragma unroll
    for (int p = 0; p < K; ++p) {
      unpack<IO, V>(rx[p], x[p]);
      if (a.gate != kGateNone) unpack<IO, V>(rz[p], z[p]);
      if (BWD) unpack<IO, V>(rd[p], d[p]);
    }
    if (row0 + per * a.nblk < a.rows) load(row0 + per * a.nblk);

    // the group's values in u, centered
    float u[K][V], s = 0.0f;
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        u[p][i] = a.gate == kGateFirst ? x[p][i] * act(a.activation, z[p][i]) : x[p][i];
        s += u[p][i];
      }
    if (a.center) {
      // divided, not multiplied by a rounded reciprocal: a group of equal values keeps no residue to be blown up
      const float mu = sum(s) / static_cast<float>(a.gs);
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) u[p][i] = in_group[p] ? u[p][i] - mu : 0.0f;
    }
    s = 0.0f;
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) s = fmaf(u[p][i], u[p][i], s);
    // 0 for the rows behind the last: with eps 0 their zeros would become NaN in the parameters' sums
    s = sum(s);
    const float r = row < a.rows ? __builtin_amdgcn_rsqf(fmaf(s, inv, a.eps)) : 0.0f;

    const int64_t out = row * a.channels;
    if (!BWD) {
#pragma unroll
      for (int p = 0; p < K; ++p) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[i] = fmaf(u[p][i] * r, w[p][i], b[p][i]);
          if (a.gate == kGateAfter) y[i] *= act(a.activation, z[p][i]);
          if (a.gate == kGateNone) y[i] = act(a.activation, y[i]);
        }
        if (in_group[p] && row < a.rows) put<IO, V>(static_cast<T*>(a.out) + out + ch[p], y);
      }
      continue;
    }
    // d becomes dxh, and z the factor of dz (gate after: dz itself)
    float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = u[p][i] * r;
        u[p][i] = xh;
        float dn = d[p][i];
        if (a.gate == kGateAfter) {
          const float n = fmaf(xh, w[p][i], b[p][i]);
          float g;
          const float da = act_grad(a.activation, z[p][i], g);
          z[p][i] = dn * n * da;
          dn *= g;
        } else if (a.gate == kGateNone) {
          float g;
          dn *= act_grad(a.activation, fmaf(xh, w[p][i], b[p][i]), g);
        }
        sw[p][i] = fmaf(dn, xh, sw[p][i]);
        sb[p][i] += dn;
        d[p][i] = dn * w[p][i];
        m1 += d[p][i];
        m2 = fmaf(d[p][i], xh, m2);
      }
    m1 = a.center ? sum(m1) * inv : 0.0f;
    m2 = sum(m2) * inv;
#pragma unroll
    for (int p = 0; p < K; ++p) {
      float dx[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dx[i] = r * (d[p][i] - m1 - u[p][i] * m2);
        if (a.gate == kGateFirst) {
          float g;
          const float da = act_grad(a.activation, z[p][i], g);
          z[p][i] = dx[i] * x[p][i] * da;
          dx[i] *= g;
        }
      }
      if (in_group[p] && row < a.rows) {
        put<IO, V>(static_cast<T*>(a.out) + out + ch[p], dx);
        if (a.gate != kGateNone) put<IO, V>(static_cast<T*>(a.dz) + out + ch[p], z[p]);
      }
    }
  }

  if (BWD && (a.pw || a.pb)) {
    // lanes that hold the same channels, then the waves, in a fixed order
    __shared__ float join[WIDE ? 1 : (kWaves - 1) * 64 * K * V];
    float* const parts[2] = {a.pw, a.pb};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!parts[q]) continue;
      float v[K][V];
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[p][i] = q == 0 ? sw[p][i] : sb[p][i];
          if (!WIDE)
            for (int o = a.ln * a.gp; o < 64; o <<= 1) v[p][i] += __shfl_xor(v[p][i], o, 64);
        }
      if (!WIDE) {
        __syncthreads();
        if (wave > 0)
#pragma unroll
          for (int p = 0; p < K; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) join[((wave - 1) * K * V + p * V + i) * 64 + lane] = v[p][i];
        __syncthreads();
        if (wave == 0)
          for (int o = 0; o < kWaves - 1; ++o)
#pragma unroll
            for (int p = 0; p < K; ++p)
#pragma unroll
              for (int i = 0; i < V; ++i) v[p][i] += join[(o * K * V + p * V + i) * 64 + lane];
      }
      if (WIDE || (wave == 0 && sub == 0))
#pragma unroll
        for (int p = 0; p < K; ++p)
          if (in_group[p])
#pragma unroll
            for (int i = 0; i < V; ++i) parts[q][static_cast<int64_t>(blk) * a.channels + ch[p] + i] = v[p][i];
    }
  }
}

// out[c] = sum over blocks of part[block][c]: 64 channels a workgroup, whose 16
// waves take every 16th block.
__global__ __launch_bounds__(1024) void gnorm_sum_kernel(int32_t nblk, int32_t channels, const float* pw,
                                                         const float* pb, float* dw, float* db) {
  __shared__ float red[16][64];
  const float* part = blockIdx.y == 0 ? pw : pb;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < channels)
    for (int j = wave; j < nblk; j += 16) s += part[static_cast<int64_t>(j) * channels + c];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < channels) {
    for (int j = 1; j < 16; ++j) s += red[j][lane];
    out[c] = s;
  }
}

// How a group is laid out over lanes.
struct Layout {
  int vec, k, threads;  // elements a piece (1: any alignment), pieces a lane, threads of a workgroup
  int ln, ln_log, gp, tiles, rp;
  bool wide;
};
Layout layout(int32_t channels, int32_t groups, int32_t io_dtype, bool can_vec) {
  Layout l{};
  const int gs = channels / groups, full = io_dtype == 0 ? 4 : 8;
  l.vec = can_vec && gs % full == 0 ? full : 1;
  const int pieces = gs / l.vec, most = l.vec == 1 ? 16 : 4;  // pieces of a lane in one wave
  l.wide = pieces > 64 * most;
  l.gp = 1;
  l.rp = 1;
  if (l.wide) {
    l.k = 16 / l.vec;
    l.threads = 256;
    while (l.threads * l.k < pieces) l.threads *= 2;
    l.ln = l.threads;
  } else {
    l.threads = 64 * kWaves;
    l.ln = 1;
    while (l.ln < 64 && l.ln < pieces) {
      l.ln *= 2;
      ++l.ln_log;
    }
    l.k = (pieces + l.ln - 1) / l.ln;
    if (l.vec == 1) l.k = l.k <= 2 ? 2 : l.k <= 8 ? 8 : 16;
    // neighbouring groups of a row, as many as divide it evenly
    while (l.gp * 2 * l.ln <= 64 && groups % (l.gp * 2) == 0) l.gp *= 2;
    l.rp = 64 / (l.ln * l.gp);
  }
  l.tiles = groups / l.gp;
  return l;
}

// Workgroups that share the rows of a tile.
int64_t blocks(const Layout& l, int64_t rows, bool bwd) {
  const int64_t per = l.wide ? 1 : static_cast<int64_t>(kWaves) * l.rp;
  const int64_t all = (rows + per - 1) / per;
  const int64_t want = ((bwd ? 1024 : 8192) + l.tiles - 1) / l.tiles;
  return all < want ? all : want;
}

template <int IO, int V, int K, bool WIDE>
hipError_t launch_typed(const GnCall& c, const Layout& l, const GnArgs& a) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(l.tiles) * a.nblk)), block(l.threads);
  if (c.dy)
    hipLaunchKernelGGL((gnorm_kernel<IO, V, K, WIDE, true>), grid, block, 0, c.stream, a);
  else
    hipLaunchKernelGGL((gnorm_kernel<IO, V, K, WIDE, false>), grid, block, 0, c.stream, a);
  return hipGetLastError();
}

template <int IO>
hipError_t launch_io(const GnCall& c, const Layout& l, const GnArgs& a) {
  constexpr int V = IO == 0 ? 4 : 8;
  if (l.wide) return l.vec == 1 ? launch_typed<IO, 1, 16, true>(c, l, a) : launch_typed<IO, V, 16 / V, true>(c, l, a);
  if (l.vec == 1) {
    if (l.k == 2) return launch_typed<IO, 1, 2, false>(c, l, a);
    return l.k == 8 ? launch_typed<IO, 1, 8, false>(c, l, a) : launch_typed<IO, 1, 16, false>(c, l, a);
  }
  switch (l.k) {
    case 1: return launch_typed<IO, V, 1, false>(c, l, a);
    case 2: return launch_typed<IO, V, 2, false>(c, l, a);
    case 3: return launch_typed<IO, V, 3, false>(c, l, a);
    default: return launch_typed<IO, V, 4, false>(c, l, a);
  }
}

}  // namespace

size_t gn_part_floats(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int sums) {
  if (sums == 0) return 0;
  // the call may take either layout, by the alignment of its tensors
  const int64_t v = blocks(layout(channels, groups, io_dtype, true), rows, true);
  const int64_t s = blocks(layout(channels, groups, io_dtype, false), rows, true);
  return static_cast<size_t>(v > s ? v : s) * channels * sums;
}

hipError_t launch_gnorm(const GnCall& c) {
  const int full = c.io_dtype == 0 ? 4 : 8;
  auto fits = [&](const void* p, int64_t row) { return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && row % full == 0; };
  const bool can_vec = fits(c.x, c.x_row) && fits(c.out, c.channels) && (!c.z || fits(c.z, c.z_row)) &&
                       (!c.dy || fits(c.dy, c.dy_row)) && (!c.dz || fits(c.dz, c.channels));
  const Layout l = layout(c.channels, c.groups, c.io_dtype, can_vec);
  GnArgs a{};
  a.rows = c.rows;
  a.x_row = c.x_row;
  a.z_row = c.z_row;
  a.dy_row = c.dy_row;
  a.channels = c.channels;
  a.gs = c.channels / c.groups;
  a.ln = l.ln;
  a.ln_log = l.ln_log;
  a.gp = l.gp;
  a.tiles = l.tiles;
  a.nblk = static_cast<int32_t>(blocks(l, c.rows, c.dy != nullptr));
  a.activation = c.activation;
  a.gate = c.gate;
  a.center = c.center;
  a.eps = c.eps;
  a.x = c.x;
  a.z = c.z;
  a.dy = c.dy;
  a.weight = c.weight;
  a.bias = c.bias;
  a.out = c.out;
  a.dz = c.dz;
  const size_t n = static_cast<size_t>(a.nblk) * c.channels;
  a.pw = c.dweight ? c.part : nullptr;
  a.pb = c.dbias ? c.part + (c.dweight ? n : 0) : nullptr;
  hipError_t e = c.io_dtype == 0 ? launch_io<0>(c, l, a) : launch_io<1>(c, l, a);
  if (e != hipSuccess || (!a.pw && !a.pb)) return e;
  hipLaunchKernelGGL(gnorm_sum_kernel, dim3(static_cast<unsigned>((c.channels + 63) / 64), 2), dim3(1024), 0, c.stream,
                     a.nblk, c.channels, a.pw, a.pb, c.dweight, c.dbias);
  return hipGetLastError();
}

}  // namespace mscan
