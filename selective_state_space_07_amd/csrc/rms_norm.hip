// RMS norm of a row (token) with the residual's addition before it, its
// gradients, and its output in 8 bits with scales.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w.
// Gradients, with hat = h r and dn = dy w:
//   dh += r (dn - hat mean(dn hat)),  dw = sum over rows of dy hat;
// dh is the gradient of x and of the residual alike.
// 8 bits: q = e4m3(y / s), s = max |y| / 448 over the row or over 128 channels.
//
// All tensors are read and written once: bound by memory traffic. A row of up to
// 1024 channels (16-byte pieces, a few a lane) is held by one wave, narrow rows
// by part of one, several side by side; a wider row by a workgroup, whose waves' sums
// meet in LDS. The row stays in registers between its sum and its output. In
// the backward lanes keep their channels from row to row, so that dw stays in
// registers and leaves as one partial sum per workgroup.
//
// Measured: forward 16384 x 768, bfloat16 with a float32 residual 26.6 us (151
// MB, 5.7 TB/s: part of it comes from the caches), its gradients 40 us (201 MB,
// 5.0 TB/s; a large copy reaches 5.2) and 7 us for the sums over workgroups;
// 4096 x 2048 with 8-bit output 11.6 us (59 MB, 5.1 TB/s); 5 x 1000 3.3 us.
#include <algorithm>
#include <type_traits>

#include "rmsnorm_internal.h"
#include "row_device.h"

namespace mscan {

namespace {

constexpr int kWaves = 4;  // waves per workgroup where a wave holds whole rows

struct RnArgs {
  int64_t rows, x_row, residual_row, h_row, dy_row, dh_row;
  int32_t channels, ln, ln_log, nblk, nscales;
  float eps;
  const void *x, *residual, *h, *dy, *dh;
  const float* weight;
  void *y, *h_out, *dx, *dresidual;
  float *scales, *pw;
};

// V elements of type R (0 float32, 1 bfloat16) as float32, V that of the io type.
template <int R, int V>
__device__ __forceinline__ void get(const void* base, int64_t at, bool ok, float (&o)[V]) {
  if constexpr (R == 0 && V == 8) {
    const float* p = static_cast<const float*>(base) + at;
    f4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
    if (ok) {
      a = *reinterpret_cast<const f4*>(p);
      b = *reinterpret_cast<const f4*>(p + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = a[i];
      o[i + 4] = b[i];
    }
  } else {
    unpack<R, V>(fetch<R, V>(base, at, ok), o);
  }
}
template <int R, int V>
__device__ __forceinline__ void set(void* base, int64_t at, const float (&o)[V]) {
  if constexpr (R == 0 && V == 8) {
    float* p = static_cast<float*>(base) + at;
    __builtin_nontemporal_store(f4{o[0], o[1], o[2], o[3]}, reinterpret_cast<f4*>(p));
    __builtin_nontemporal_store(f4{o[4], o[5], o[6], o[7]}, reinterpret_cast<f4*>(p + 4));
  } else {
    put<R, V>(static_cast<typename Io<R>::T*>(base) + at, o);
  }
}

// Of absolute values as their bits, so that a NaN is the largest: the maximum
// over the 1 to 64 lanes of a group, in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int ln) {
  if (ln > 1) v = dpp_max<0xB1>(v);
  if (ln > 2) v = dpp_max<0x4E>(v);
  if (ln > 4) v = dpp_max<0x141>(v);
  if (ln > 8) v = dpp_max<0x140>(v);
  if (ln > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = r[0] > r[1] ? r[0] : r[1];
  }
  if (ln > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = r[0] > r[1] ? r[0] : r[1];
  }
  return v;
}
// The scale of a block whose largest absolute value has these bits.
__device__ __forceinline__ float scale_of(uint32_t most) {
  const float s = __uint_as_float(most) / 448.0f;
  return most == 0 ? 1.0f : s < 0x1p-126f ? 0x1p-126f : s;
}
template <int V>
__device__ __forceinline__ void put8(void* base, int64_t at, const float (&q)[V]) {
  int w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w[i], true);
  }
  char* p = static_cast<char*>(base) + at;
  if constexpr (V == 8)
    *reinterpret_cast<u2*>(p) = u2{static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[1])};
  else
    *reinterpret_cast<int*>(p) = w[0];
}

// A lane's place in its row, the sum over the row, and the row's scale.
template <int V, int K, bool WIDE, int N>
struct Row {
  int in, sub, lanes, half = 0;
  bool has[K];
  int ch[K];
  float (*red)[N][16];
  __device__ __forceinline__ Row(const RnArgs& a, float (*red_)[N][16]) : red(red_) {
    const int lane = threadIdx.x & 63;
    in = WIDE ? static_cast<int>(threadIdx.x) : lane & (a.ln - 1);
    sub = WIDE ? 0 : lane >> a.ln_log;
    lanes = !WIDE ? a.ln : V == 1 && K == 16 ? 1024 : static_cast<int>(blockDim.x);  // a constant: the pieces' places are one's
#pragma unroll
    for (int p = 0; p < K; ++p) {
      ch[p] = (p * lanes + in) * V;
      has[p] = ch[p] < a.channels;
    }
  }
  __device__ __forceinline__ float sum(float v) {
    if constexpr (!WIDE) {
      return lanes_sum(v, lanes);
    } else {
      float w[N] = {v};
      wide_sum(w, *reinterpret_cast<float(*)[2][N][16]>(red), half);
      half ^= 1;
      return w[0];
    }
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = lanes_max(v, WIDE ? 64 : lanes);
    if constexpr (WIDE) {
      if ((threadIdx.x & 63) == 0) red[half][0][threadIdx.x >> 6] = __uint_as_float(v);
      __syncthreads();
      for (int w = 0; w < lanes >> 6; ++w) {
        const uint32_t o = __float_as_uint(red[half][0][w]);
        v = v > o ? v : o;
      }
      half ^= 1;
    }
    return v;
  }
  // Takes h, and gives it times `scale` (1 almost always) with 1 / sqrt(..) of that.
  __device__ __forceinline__ float root(const RnArgs& a, float (&h)[K][V], float& scale, bool live) {
    const float inv = 1.0f / static_cast<float>(a.channels);
    auto squares = [&]() {
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(h[p][i], h[p][i], s);
      return sum(s);
    };
    float s = squares();
    scale = scale_for(s, fmaf(s, inv, a.eps));
    if (__any(scale != 1.0f)) {  // the same for all of a workgroup that shares a row
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) h[p][i] *= scale;
      s = squares();
      if (s == 0.0f) scale = 1.0f;
    }
    return live ? __builtin_amdgcn_rsqf(fmaf(s, inv, a.eps * scale * scale)) : 0.0f;
  }
};

// OUT: 0 the io type, 1 one 8-bit scale a row, 2 one for 128 channels.
template <int IO, int R, int V, int K, bool WIDE, int OUT>
__global__ __launch_bounds__(WIDE ? 1024 : 64 * kWaves) void rms_fwd_kernel(const RnArgs a) {
  __shared__ float red[2][1][WIDE ? 16 : 1];
  Row<V, K, WIDE, 1> row(a, reinterpret_cast<float(*)[1][16]>(red));
  const int rp = WIDE ? 1 : 64 >> a.ln_log;  // rows side by side in a wave
  const int64_t per = WIDE ? 1 : kWaves * rp;
  float w[K][V];
#pragma unroll
  for (int p = 0; p < K; ++p) fetch_params<V>(a.weight, row.ch[p], row.has[p], 1.0f, w[p]);
  for (int64_t r0 = blockIdx.x * per; r0 < a.rows; r0 += per * a.nblk) {
    const int64_t r = WIDE ? r0 : r0 + static_cast<int64_t>(threadIdx.x >> 6) * rp + row.sub;
    const bool live = r < a.rows;
    float h[K][V];
#pragma unroll
    for (int p = 0; p < K; ++p) get<IO, V>(a.x, r * a.x_row + row.ch[p], live && row.has[p], h[p]);
    if (a.residual) {
      float q[K][V];
#pragma unroll
      for (int p = 0; p < K; ++p) get<R, V>(a.residual, r * a.residual_row + row.ch[p], live && row.has[p], q[p]);
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) h[p][i] += q[p][i];
    }
    const int64_t at = r * a.channels;
    if (a.h_out)
#pragma unroll
      for (int p = 0; p < K; ++p)
        if (live && row.has[p]) set<R, V>(a.h_out, at + row.ch[p], h[p]);
    float scale;
    const float root = row.root(a, h, scale, live);
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) h[p][i] *= root * w[p][i];
    if constexpr (OUT == 0) {
#pragma unroll
      for (int p = 0; p < K; ++p)
        if (live && row.has[p]) set<IO, V>(a.y, at + row.ch[p], h[p]);
    } else {
      uint32_t most[K];
#pragma unroll
      for (int p = 0; p < K; ++p) {
        most[p] = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t u = row.has[p] ? __float_as_uint(h[p][i]) & 0x7FFFFFFFu : 0;
          most[p] = most[p] > u ? most[p] : u;
        }
        if constexpr (OUT == 2) most[p] = lanes_max(most[p], row.lanes < 128 / V ? row.lanes : 128 / V);
      }
      if constexpr (OUT == 1) {
        uint32_t m = most[0];
#pragma unroll
        for (int p = 1; p < K; ++p) m = m > most[p] ? m : most[p];
        m = row.max(m);
#pragma unroll
        for (int p = 0; p < K; ++p) most[p] = m;
      }
#pragma unroll
      for (int p = 0; p < K; ++p) {
        if (!live || !row.has[p]) continue;
        const float s = scale_of(most[p]), inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < V; ++i) h[p][i] *= inv;
        put8<V>(a.y, at + row.ch[p], h[p]);
        if (OUT == 1 ? row.ch[p] == 0 : row.ch[p] % 128 == 0) a.scales[r * a.nscales + (OUT == 1 ? 0 : row.ch[p] / 128)] = s;
      }
    }
  }
}

template <int IO, int R, int V, int K, bool WIDE>
__global__ __launch_bounds__(WIDE ? 1024 : 64 * kWaves) void rms_bwd_kernel(const RnArgs a) {
  __shared__ float red[2][1][WIDE ? 16 : 1];
  Row<V, K, WIDE, 1> row(a, reinterpret_cast<float(*)[1][16]>(red));
  const int rp = WIDE ? 1 : 64 >> a.ln_log;
  const int64_t per = WIDE ? 1 : kWaves * rp;
  const float inv = 1.0f / static_cast<float>(a.channels);
  // sixteen single elements a thread of 1024, 128 registers each, leave room for h and dw alone: the others are read where
  // they are used, piece by piece
  constexpr bool kHeld = !(WIDE && V == 1 && K == 16);
  float w[kHeld ? K : 1][V], sw[K][V];
#pragma unroll
  for (int p = 0; p < K; ++p) {
    if constexpr (kHeld) fetch_params<V>(a.weight, row.ch[p], row.has[p], 1.0f, w[p]);
#pragma unroll
    for (int i = 0; i < V; ++i) sw[p][i] = 0.0f;
  }
  for (int64_t r0 = blockIdx.x * per; r0 < a.rows; r0 += per * a.nblk) {
    const int64_t r = WIDE ? r0 : r0 + static_cast<int64_t>(threadIdx.x >> 6) * rp + row.sub;
    const bool live = r < a.rows;
    float h[K][V], d[kHeld ? K : 1][V], back[kHeld ? K : 1][V];
    // dy (or, `from` dh) of a piece, and not before its use
    auto again = [&](int p, auto from, float (&o)[V]) {
      int t = row.ch[p];
      asm volatile("" : "+v"(t)::"memory");
      if constexpr (decltype(from)::value)
        get<R, V>(a.dh, r * a.dh_row + t, live && row.has[p] && a.dh, o);
      else
        get<IO, V>(a.dy, r * a.dy_row + t, live && row.has[p], o);
    };
#pragma unroll
    for (int p = 0; p < K; ++p) {
      const bool ok = live && row.has[p];
      int from = row.ch[p];
      if constexpr (!kHeld) asm volatile("" : "+v"(from));
      get<R, V>(a.h, r * a.h_row + from, ok, h[p]);
      if constexpr (kHeld) {
        get<IO, V>(a.dy, r * a.dy_row + row.ch[p], ok, d[p]);
        get<R, V>(a.dh, r * a.dh_row + row.ch[p], ok && a.dh, back[p]);
      }
    }
    float scale;
    const float root = row.root(a, h, scale, live);
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < K; ++p) {
      float(&dp)[V] = d[kHeld ? p : 0];
      if constexpr (!kHeld) {
        again(p, std::false_type{}, dp);
        fetch_params<V>(a.weight, row.ch[p], row.has[p], 1.0f, w[0]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[p][i] *= root;  // hat
        sw[p][i] = fmaf(dp[i], h[p][i], sw[p][i]);
        dp[i] *= w[kHeld ? p : 0][i];
        m = fmaf(dp[i], h[p][i], m);
      }
    }
    m = row.sum(m) * inv;
    const float slope = root * scale;
    const int64_t at = r * a.channels;
#pragma unroll
    for (int p = 0; p < K; ++p) {
      float(&dp)[V] = d[kHeld ? p : 0];
      if constexpr (!kHeld) {
        again(p, std::false_type{}, dp);
        again(p, std::true_type{}, back[0]);
        fetch_params<V>(a.weight, row.ch[p], row.has[p], 1.0f, w[0]);
#pragma unroll
        for (int i = 0; i < V; ++i) dp[i] *= w[0][i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) dp[i] = fmaf(slope, fmaf(-h[p][i], m, dp[i]), back[kHeld ? p : 0][i]);
      int to = row.ch[p];
      if constexpr (!kHeld) asm volatile("" : "+v"(to));
      if (live && row.has[p]) {
        if (a.dresidual) set<R, V>(a.dresidual, at + to, dp);
        if (a.dx) set<IO, V>(a.dx, at + to, dp);
      }
    }
  }
  if (!a.pw) return;
  // lanes that hold the same channels, then the waves, in a fixed order
  if constexpr (!WIDE) {
    __shared__ float join[(kWaves - 1) * 64 * K * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        for (int o = a.ln; o < 64; o <<= 1) sw[p][i] += __shfl_xor(sw[p][i], o, 64);
        if (wave > 0) join[((wave - 1) * K * V + p * V + i) * 64 + lane] = sw[p][i];
      }
    __syncthreads();
    if (wave > 0 || row.sub > 0) return;
    for (int o = 0; o < kWaves - 1; ++o)
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) sw[p][i] += join[(o * K * V + p * V + i) * 64 + lane];
  }
#pragma unroll
  for (int p = 0; p < K; ++p)
    if (row.has[p])
#pragma unroll
      for (int i = 0; i < V; ++i) a.pw[static_cast<int64_t>(blockIdx.x) * a.channels + row.ch[p] + i] = sw[p][i];
}

// How a row is laid out over lanes.
struct Layout {
  int vec, k, threads, ln, ln_log;
  bool wide;
};
Layout layout(int32_t channels, int32_t io_dtype, bool can_vec) {
  Layout l{};
  const int full = io_dtype == 0 ? 4 : 8;
  l.vec = can_vec && channels % full == 0 ? full : 1;
  const int pieces = channels / l.vec, most = l.vec == 1 ? 8 : io_dtype == 0 ? 4 : 2;  // pieces of a lane in one wave
  l.wide = pieces > 64 * most;
  if (l.wide) {
    l.k = l.vec == 1 ? (pieces <= 4096 ? 4 : 16) : pieces <= 1024 ? 1 : io_dtype == 0 ? 4 : 2;
    l.threads = l.k == 16 ? 1024 : ((pieces + l.k - 1) / l.k + 63) / 64 * 64;
    l.ln = l.threads;
  } else {
    l.threads = 64 * kWaves;
    l.ln = 1;
    while (l.ln < 64 && l.ln < pieces) {
      l.ln *= 2;
      ++l.ln_log;
    }
    l.k = l.vec == 1 ? 8 : pieces <= 64 ? 1 : pieces <= 128 ? 2 : 4;
    if (l.vec == 1 && pieces <= 64) l.k = 1;
  }
  return l;
}

int64_t blocks(const Layout& l, int64_t rows, bool bwd) {
  const int64_t per = l.wide ? 1 : kWaves * (64 / l.ln), all = (rows + per - 1) / per;
  // (a dispatch dimension counts its work-items in 32 bits)
  const int64_t most = bwd ? 256 * (l.wide ? std::max(1, 1024 / l.threads) : 4) : std::min(int64_t{1} << 22, (int64_t{1} << 31) / l.threads);
  const int64_t turns = (all + most - 1) / most;
  return (all + turns - 1) / turns;
}

template <int IO, int R, int V, int K, bool WIDE>
hipError_t launch_typed(const RnCall& c, const Layout& l, const RnArgs& a) {
  const dim3 grid(static_cast<unsigned>(a.nblk)), block(l.threads);
  if (c.dy) {
    hipLaunchKernelGGL((rms_bwd_kernel<IO, R, V, K, WIDE>), grid, block, 0, c.stream, a);
  } else if (!c.scales) {
    hipLaunchKernelGGL((rms_fwd_kernel<IO, R, V, K, WIDE, 0>), grid, block, 0, c.stream, a);
  } else if constexpr (V > 1) {
    if (c.block == 0)
      hipLaunchKernelGGL((rms_fwd_kernel<IO, R, V, K, WIDE, 1>), grid, block, 0, c.stream, a);
    else
      hipLaunchKernelGGL((rms_fwd_kernel<IO, R, V, K, WIDE, 2>), grid, block, 0, c.stream, a);
  } else {
    return hipErrorInvalidValue;  // 8-bit outputs are written by pieces alone
  }
  return hipGetLastError();
}

template <int IO, int R>
hipError_t launch_io(const RnCall& c, const Layout& l, const RnArgs& a) {
  constexpr int V = IO == 0 ? 4 : 8, kMost = IO == 0 ? 4 : 2;
  if (l.vec == 1) {
    if (!l.wide) return l.k == 1 ? launch_typed<IO, R, 1, 1, false>(c, l, a) : launch_typed<IO, R, 1, 8, false>(c, l, a);
    return l.k == 4 ? launch_typed<IO, R, 1, 4, true>(c, l, a) : launch_typed<IO, R, 1, 16, true>(c, l, a);
  }
  if (l.wide) return l.k == 1 ? launch_typed<IO, R, V, 1, true>(c, l, a) : launch_typed<IO, R, V, kMost, true>(c, l, a);
  if (l.k == 1) return launch_typed<IO, R, V, 1, false>(c, l, a);
  return l.k == 2 ? launch_typed<IO, R, V, 2, false>(c, l, a) : launch_typed<IO, R, V, kMost, false>(c, l, a);
}

}  // namespace

size_t rn_part_floats(int64_t rows, int32_t channels, int32_t io_dtype) {
  // the call may take either layout, by the alignment of its tensors
  const int64_t v = blocks(layout(channels, io_dtype, true), rows, true);
  const int64_t s = blocks(layout(channels, io_dtype, false), rows, true);
  return static_cast<size_t>(v > s ? v : s) * channels;
}

hipError_t launch_rmsnorm(const RnCall& c) {
  // 16 bytes of each tensor's own type: a piece of eight bfloat16 channels meets a float32 residual as two of four (16384 x
  // 768, residual rows 772 apart: forward 28 us, gradients 38; by single elements, as where they start off 16 bytes, 36 and 58)
  const int64_t es = c.io_dtype == 0 ? 4 : 2, rs = c.residual_dtype == 0 ? 4 : 2;
  auto fits = [](const void* p, int64_t row_bytes) { return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0); };
  const bool can_vec = fits(c.x, c.x_row * es) && fits(c.residual, c.residual_row * rs) && fits(c.h, c.h_row * rs) &&
                       fits(c.dy, c.dy_row * es) && fits(c.dh, c.dh_row * rs) && fits(c.y, 0) && fits(c.h_out, 0) &&
                       fits(c.dx, 0) && fits(c.dresidual, 0);
  const Layout l = layout(c.channels, c.io_dtype, can_vec);
  RnArgs a{};
  a.rows = c.rows;
  a.x_row = c.x_row;
  a.residual_row = c.residual_row;
  a.h_row = c.h_row;
  a.dy_row = c.dy_row;
  a.dh_row = c.dh_row;
  a.channels = c.channels;
  a.ln = l.ln;
  a.ln_log = l.ln_log;
  a.nblk = static_cast<int32_t>(blocks(l, c.rows, c.dy != nullptr));
  a.nscales = c.block ? (c.channels + c.block - 1) / c.block : 1;
  a.eps = c.eps;
  a.x = c.x;
  a.residual = c.residual;
  a.h = c.h;
  a.dy = c.dy;
  a.dh = c.dh;
  a.weight = c.weight;
  a.y = c.y;
  a.h_out = c.h_out;
  a.dx = c.dx;
  a.dresidual = c.dresidual;
  a.scales = c.scales;
  a.pw = c.dweight ? c.part : nullptr;
  hipError_t e;
  if (c.io_dtype == 0)
    e = launch_io<0, 0>(c, l, a);
  else
    e = c.residual_dtype == 0 ? launch_io<1, 0>(c, l, a) : launch_io<1, 1>(c, l, a);
  if (e != hipSuccess || !a.pw) return e;
  return launch_part_sums(a.nblk, {{c.channels, a.pw, c.dweight}}, c.stream);
}

}  // namespace mscan
