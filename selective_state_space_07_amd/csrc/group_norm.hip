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
// memory traffic, and by how much of it is under way. A group of up to 512
// bytes' worth of 16-byte pieces, one a lane, is held by 1 to 64 lanes of one
// wave, which takes several neighbouring groups and several rows at a time; a
// larger one by a workgroup of up to 16 waves, one piece a lane,
// whose waves' sums meet in LDS (the largest are read anew instead; a wave that held all of 1536 channels would
// need 300 registers in the backward and leave its SIMD with one wave). The
// mean is taken first and the squares of what is left of it, in float32.
// Lanes keep their channels from row to row, so that the sums over rows stay
// in registers and leave as one partial sum per workgroup, which a second
// kernel adds in a fixed order.
//
// Measured on an MI355X, where a large copy reaches 5.2 TB/s: 16384 x 1536
// bfloat16, 12 groups, gate behind: 30 us (151 MB, 5.0 TB/s; 64 us with the gate
// chosen at each element and one row at a time). Gradients of one group, RMS,
// gate first: 60 us (252 MB, 4.2 TB/s: the sums meet twice a row, and what is
// resident waits for them; 132 us with a wave to a row).
#include "gnorm_internal.h"
#include "row_device.h"

namespace mscan {

namespace {

constexpr int kWaves = 4;            // waves per workgroup where a wave holds whole groups
constexpr int kGateNone = 0, kGateAfter = 1, kGateFirst = 2, kGateAny = 3;

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

// V elements a piece, K pieces a lane, U rows at a time. WIDE: one group of
// one row per workgroup. GATE: one of the three, or kGateAny where the call says.
// With that the gradients of eight pieces spill, or leave a SIMD two waves (16384
// x 1500 bf16, five groups, gate first: 267 us, 127 us with the gate compiled in).
template <int IO, int V, int K, int U, bool WIDE, bool BWD, int GATE>
__global__ __launch_bounds__(WIDE ? 1024 : 64 * kWaves) void gnorm_kernel(const GnArgs a) {
  using T = typename Io<IO>::T;
  const int gate_kind = GATE == kGateAny ? a.gate : GATE;
  static_assert(!WIDE || U == 1, "a workgroup's sums meet row by row");
  __shared__ float red[2][2][WIDE ? 16 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x % a.tiles, blk = blockIdx.x / a.tiles;
  const int in = WIDE ? tid : lane & (a.ln - 1);              // lane within its group
  const int slot = WIDE ? 0 : lane >> a.ln_log;               // which of the wave's groups
  const int sub = WIDE ? 0 : slot / a.gp;                     // which of the wave's rows
  const int rp = WIDE ? 1 : 64 / (a.ln * a.gp);               // rows side by side in a wave
  const int ch0 = (tile * a.gp + (slot - sub * a.gp)) * a.gs;  // the group's first channel
  const int lanes = WIDE ? static_cast<int>(blockDim.x) : a.ln;
  const float inv = 1.0f / static_cast<float>(a.gs);
  int half = 0;
  auto sum = [&](float (&v)[2]) {  // over the group, in all of its lanes
    if constexpr (WIDE) {
      wide_sum(v, red, half);
      half ^= 1;
    } else {
      v[0] = lanes_sum(v[0], a.ln);
      v[1] = lanes_sum(v[1], a.ln);
    }
  };
  auto sum1 = [&](float v) {
    float w[2] = {v, 0.0f};
    if constexpr (WIDE) {
      sum(w);
      return w[0];
    } else {
      return lanes_sum(v, a.ln);
    }
  };

  int ch[K];
  bool in_group[K];
  float w[K][V], b[K][V], sw[BWD ? K : 1][V], sb[BWD ? K : 1][V];
#pragma unroll
  for (int p = 0; p < K; ++p) {
    const int e = (p * lanes + in) * V;
    in_group[p] = e < a.gs;
    ch[p] = ch0 + e;
    fetch_params<V>(a.weight, ch[p], in_group[p], 1.0f, w[p]);
    fetch_params<V>(a.bias, ch[p], in_group[p], 0.0f, b[p]);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (BWD) sw[p][i] = sb[p][i] = 0.0f;
  }

  const int64_t per = WIDE ? 1 : static_cast<int64_t>(kWaves) * U * rp;  // rows of a workgroup at a time
  int64_t row0 = blk * per + (WIDE ? 0 : static_cast<int64_t>(wave) * U * rp);  // uniform in the wave
  Vec<IO, V> rx[U][K], rz[U][K], rd[BWD ? U : 1][K];
  auto load = [&](int64_t r0) {
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int p = 0; p < K; ++p) {
        const int64_t row = r0 + q * rp + sub;
        const bool ok = in_group[p] && row < a.rows;
        rx[q][p] = fetch<IO, V>(a.x, row * a.x_row + ch[p], ok);
        if (gate_kind != kGateNone) rz[q][p] = fetch<IO, V>(a.z, row * a.z_row + ch[p], ok);
        if (BWD) rd[q][p] = fetch<IO, V>(a.dy, row * a.dy_row + ch[p], ok);
      }
  };
  for (; row0 < a.rows; row0 += per * a.nblk) {
    load(row0);
    float x[U][K][V], z[U][K][V], d[BWD ? U : 1][K][V], gate[BWD ? U : 1][K][V], u[U][K][V], r[U], rdx[U];
#pragma unroll
    for (int q = 0; q < U; ++q)
#pragma unroll
      for (int p = 0; p < K; ++p) {
        unpack<IO, V>(rx[q][p], x[q][p]);
        if (gate_kind != kGateNone) unpack<IO, V>(rz[q][p], z[q][p]);
        if (BWD) unpack<IO, V>(rd[q][p], d[q][p]);
      }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      // the group's values in u, centered
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          u[q][p][i] = x[q][p][i];
          if (gate_kind == kGateFirst) {
            float g;
            if (BWD) {  // z becomes the derivative, the gate itself is kept too
              z[q][p][i] = act_grad(a.activation, z[q][p][i], g);
              gate[q][p][i] = g;
            } else {
              g = act(a.activation, z[q][p][i]);
            }
            u[q][p][i] *= g;
          }
          s += u[q][p][i];
        }
      auto statistics = [&]() {  // of u, whose sum is s: its mean taken off, the sum of its squares
        if (a.center) {
          // divided, not multiplied by a rounded reciprocal: a group of equal values keeps no residue to be blown up
          const float mu = sum1(s) / static_cast<float>(a.gs);
#pragma unroll
          for (int p = 0; p < K; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) u[q][p][i] = in_group[p] ? u[q][p][i] - mu : 0.0f;
        }
        s = 0.0f;
#pragma unroll
        for (int p = 0; p < K; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i) s = fmaf(u[q][p][i], u[q][p][i], s);
        s = sum1(s);
      };
      statistics();
      float scale = scale_for(s, fmaf(s, inv, a.eps));
      if (__any(scale != 1.0f)) {  // the same for all of a workgroup that shares a group
        s = 0.0f;
#pragma unroll
        for (int p = 0; p < K; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            u[q][p][i] = x[q][p][i] * scale;
            if (gate_kind == kGateFirst) u[q][p][i] *= BWD ? gate[q][p][i] : act(a.activation, z[q][p][i]);
            s += u[q][p][i];
          }
        statistics();
        if (s == 0.0f) scale = 1.0f;
        if (BWD && gate_kind == kGateFirst)  // these are what dx and dz take of it
#pragma unroll
          for (int p = 0; p < K; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[q][p][i] *= scale;
              gate[q][p][i] *= scale;
            }
      }
      // 0 for the rows behind the last: with eps 0 their zeros would become NaN in the parameters' sums
      r[q] = row0 + q * rp + sub < a.rows ? __builtin_amdgcn_rsqf(fmaf(s, inv, a.eps * scale * scale)) : 0.0f;
      rdx[q] = gate_kind == kGateFirst ? r[q] : r[q] * scale;
    }

#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t row = row0 + q * rp + sub, out = row * a.channels;
      if (!BWD) {
#pragma unroll
        for (int p = 0; p < K; ++p) {
          float y[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            y[i] = fmaf(u[q][p][i] * r[q], w[p][i], b[p][i]);
            if (gate_kind == kGateAfter) y[i] *= act(a.activation, z[q][p][i]);
            if (gate_kind == kGateNone) y[i] = act(a.activation, y[i]);
          }
          if (in_group[p] && row < a.rows) put<IO, V>(static_cast<T*>(a.out) + out + ch[p], y);
        }
        continue;
      }
      // d becomes dxh, and z the factor of dz (gate after: dz itself)
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < K; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = u[q][p][i] * r[q];
          u[q][p][i] = xh;
          float dn = d[q][p][i];
          if (gate_kind == kGateAfter) {
            const float n = fmaf(xh, w[p][i], b[p][i]);
            float g;
            const float da = act_grad(a.activation, z[q][p][i], g);
            z[q][p][i] = dn * n * da;
            dn *= g;
          } else if (gate_kind == kGateNone) {
            float g;
            dn *= act_grad(a.activation, fmaf(xh, w[p][i], b[p][i]), g);
          }
          sw[p][i] = fmaf(dn, xh, sw[p][i]);
          sb[p][i] += dn;
          d[q][p][i] = dn * w[p][i];
          m[0] += d[q][p][i];
          m[1] = fmaf(d[q][p][i], xh, m[1]);
        }
      sum(m);
      const float m1 = a.center ? m[0] * inv : 0.0f, m2 = m[1] * inv;
#pragma unroll
      for (int p = 0; p < K; ++p) {
        float dx[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dx[i] = rdx[q] * (d[q][p][i] - m1 - u[q][p][i] * m2);
          if (gate_kind == kGateFirst) {
            z[q][p][i] *= dx[i] * x[q][p][i];
            dx[i] *= gate[q][p][i];
          }
        }
        if (in_group[p] && row < a.rows) {
          put<IO, V>(static_cast<T*>(a.out) + out + ch[p], dx);
          if (gate_kind != kGateNone) put<IO, V>(static_cast<T*>(a.dz) + out + ch[p], z[q][p]);
        }
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

// A group of more values than one piece (4 single elements) a thread, 16 at the
// most: it is not kept. Every pass reads it again, from the caches (a row of
// three such tensors is at most 192 KB), piece by piece, and only the sums over
// rows stay in registers. Held whole, a lane's values left 300 to 750 bytes in
// scratch memory: gradients of 1024 x 16384, one group, 151 us in bfloat16 and
// 230 in float32, 95 and 133 so; forward 33 and 47 us, 31 and 66 so.
template <int IO, int V, bool BWD>
__global__ __launch_bounds__(1024) void gnorm_large_kernel(const GnArgs a) {
  using T = typename Io<IO>::T;
  constexpr int K = 16 / V;
  __shared__ float red[2][2][16];
  const int lanes = static_cast<int>(blockDim.x);
  const int ch0 = static_cast<int>(blockIdx.x % a.tiles) * a.gs, blk = blockIdx.x / a.tiles;
  const float inv = 1.0f / static_cast<float>(a.gs);
  int half = 0;
  auto sum = [&](float v0, float v1, float (&v)[2]) {
    v[0] = v0;
    v[1] = v1;
    wide_sum(v, red, half);
    half ^= 1;
  };
  float sw[BWD ? K : 1][V], sb[BWD ? K : 1][V];
  if constexpr (BWD) {
#pragma unroll
    for (int p = 0; p < K; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) sw[p][i] = sb[p][i] = 0.0f;
  }
  // f(piece, first channel of the group) for the thread's pieces, one by one
  auto pieces = [&](auto&& f) {
#pragma unroll
    for (int p = 0; p < K; ++p) {
      int t = threadIdx.x;
      asm volatile("" : "+v"(t)::"memory");  // its places and loads not before the last piece's use
      const int e = (p * lanes + t) * V;
      if (e < a.gs) f(p, e);
    }
  };
  for (int64_t row = blk; row < a.rows; row += a.nblk) {
    const int64_t at_x = row * a.x_row + ch0, at_z = row * a.z_row + ch0, at_dy = row * a.dy_row + ch0;
    const int64_t out = row * a.channels + ch0;
    float scale = 1.0f;
    // the values of a piece before their norm (gated, where the gate is first)
    auto read = [&](int e, float (&x)[V], float (&z)[V], float (&u)[V]) {
      unpack<IO, V>(fetch<IO, V>(a.x, at_x + e, true), x);
      if (a.gate != kGateNone) unpack<IO, V>(fetch<IO, V>(a.z, at_z + e, true), z);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = scale * (a.gate == kGateFirst ? x[i] * act(a.activation, z[i]) : x[i]);
    };
    float x[V], z[V], u[V], v[2], mu = 0.0f, t = 0.0f;
    for (int turn = 0; turn < 2; ++turn) {
      if (a.center) {
        t = 0.0f;
        pieces([&](int, int e) {
          read(e, x, z, u);
#pragma unroll
          for (int i = 0; i < V; ++i) t += u[i];
        });
        sum(t, 0.0f, v);
        mu = v[0] / static_cast<float>(a.gs);  // divided: see above
      }
      t = 0.0f;
      pieces([&](int, int e) {
        read(e, x, z, u);
#pragma unroll
        for (int i = 0; i < V; ++i) t = fmaf(u[i] - mu, u[i] - mu, t);
      });
      sum(t, 0.0f, v);
      if (turn == 0) scale = scale_for(v[0], fmaf(v[0], inv, a.eps));  // the same for all threads
      if (scale == 1.0f) break;
    }
    const float less = v[0] == 0.0f ? 1.0f : scale, r = __builtin_amdgcn_rsqf(fmaf(v[0], inv, a.eps * less * less));
    float w[V], b[V];
    if constexpr (!BWD) {
      pieces([&](int, int e) {
        read(e, x, z, u);
        fetch_params<V>(a.weight, ch0 + e, true, 1.0f, w);
        fetch_params<V>(a.bias, ch0 + e, true, 0.0f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          u[i] = fmaf((u[i] - mu) * r, w[i], b[i]);
          if (a.gate == kGateAfter) u[i] *= act(a.activation, z[i]);
          if (a.gate == kGateNone) u[i] = act(a.activation, u[i]);
        }
        put<IO, V>(static_cast<T*>(a.out) + out + e, u);
      });
    } else {
      // u becomes xh, d becomes dn, and z the factor of dz (gate after: dz itself)
      float d[V];
      auto grads = [&](int e) {
        read(e, x, z, u);
        unpack<IO, V>(fetch<IO, V>(a.dy, at_dy + e, true), d);
        fetch_params<V>(a.weight, ch0 + e, true, 1.0f, w);
        fetch_params<V>(a.bias, ch0 + e, true, 0.0f, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          u[i] = (u[i] - mu) * r;
          if (a.gate == kGateFirst) continue;
          const float n = fmaf(u[i], w[i], b[i]);
          float g;
          const float da = act_grad(a.activation, a.gate == kGateNone ? n : z[i], g);
          if (a.gate == kGateAfter) z[i] = d[i] * n * da;
          d[i] *= a.gate == kGateNone ? da : g;
        }
      };
      float m0 = 0.0f, m1 = 0.0f;
      pieces([&](int p, int e) {
        grads(e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sw[p][i] = fmaf(d[i], u[i], sw[p][i]);
          sb[p][i] += d[i];
          m0 = fmaf(d[i], w[i], m0);
          m1 = fmaf(d[i] * w[i], u[i], m1);
        }
      });
      sum(m0, m1, v);
      m0 = a.center ? v[0] * inv : 0.0f;
      m1 = v[1] * inv;
      pieces([&](int, int e) {
        grads(e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] = r * (d[i] * w[i] - m0 - u[i] * m1);
          if (a.gate == kGateFirst) {
            float g;
            z[i] = act_grad(a.activation, z[i], g) * d[i] * (x[i] * less);
            d[i] *= g;
          }
          d[i] *= less;
        }
        put<IO, V>(static_cast<T*>(a.out) + out + e, d);
        if (a.gate != kGateNone) put<IO, V>(static_cast<T*>(a.dz) + out + e, z);
      });
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int p = 0; p < K; ++p) {
      const int e = (p * lanes + static_cast<int>(threadIdx.x)) * V;
      if (e >= a.gs) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int64_t at = static_cast<int64_t>(blk) * a.channels + ch0 + e + i;
        if (a.pw) a.pw[at] = sw[p][i];
        if (a.pb) a.pb[at] = sb[p][i];
      }
    }
  }
}

// How a group is laid out over lanes.
struct Layout {
  int vec, k, u, threads;  // elements a piece (1: any alignment), pieces a lane, rows at a time, threads of a workgroup
  int ln, ln_log, gp, tiles, rp;
  bool wide;
};
Layout layout(int32_t channels, int32_t groups, int32_t io_dtype, bool can_vec, bool bwd) {
  Layout l{};
  const int gs = channels / groups, full = io_dtype == 0 ? 4 : 8;
  l.vec = can_vec && gs % full == 0 ? full : 1;
  const int pieces = gs / l.vec, most = l.vec == 1 ? 8 : 1;  // pieces of a lane in one wave
  l.wide = pieces > 64 * most;
  l.gp = 1;
  l.rp = 1;
  l.u = 1;
  if (l.wide) {
    // whole waves, of as few pieces a lane as 16 of them allow; 16 values a lane: gnorm_large_kernel
    l.k = l.vec == 1 ? (pieces <= 4096 ? 4 : 16) : pieces <= 1024 ? 1 : io_dtype == 0 ? 4 : 2;
    l.threads = ((pieces + l.k - 1) / l.k + 63) / 64 * 64;
    l.ln = l.threads;
  } else {
    l.threads = 64 * kWaves;
    l.ln = 1;
    while (l.ln < 64 && l.ln < pieces) {
      l.ln *= 2;
      ++l.ln_log;
    }
    l.k = (pieces + l.ln - 1) / l.ln;
    if (l.vec == 1) l.k = l.k <= 2 ? 2 : 8;
    if (l.vec > 1) l.u = bwd ? 2 : 4;
    // neighbouring groups of a row, as many as divide it evenly
    while (l.gp * 2 * l.ln <= 64 && groups % (l.gp * 2) == 0) l.gp *= 2;
    l.rp = 64 / (l.ln * l.gp);
  }
  l.tiles = groups / l.gp;
  return l;
}

// Workgroups that share the rows of a tile, with as many turns for each. The
// backward takes about one round of what is resident, so that few partial sums
// are left: 16 waves on a CU (float32: 24), or three workgroups of four waves
// where a wave holds whole groups (16384 x 1536 bf16, one group, three waves:
// 1280 workgroups 60 us, 1536 71 us, 768 69 us). Three are a round and a half
// for the gate-first form, of which 181 registers let two be resident, and the
// best for it all the same (twelve groups, bf16, two, three and four a CU: gate
// first 68, 56 and 60 us, gate behind 54, 47 and 50, none 48, 39 and 41).
int64_t blocks(const Layout& l, int64_t rows, int32_t io_dtype, bool bwd) {
  const int64_t per = l.wide ? 1 : static_cast<int64_t>(kWaves) * l.u * l.rp;
  const int64_t all = (rows + per - 1) / per;
  const int waves = l.threads / 64, held = (io_dtype == 0 ? 24 : 16) / waves;
  const int64_t slots = 256 * (!l.wide ? 3 : held > 1 ? held : 1);
  const int64_t most = ((bwd ? slots : 16384) + l.tiles - 1) / l.tiles;
  const int64_t turns = (all + most - 1) / most;
  return (all + turns - 1) / turns;
}

template <int IO, int V, int K, int UF, int UB, bool WIDE, int GATE>
hipError_t launch_gate(const GnCall& c, const Layout& l, const GnArgs& a) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(l.tiles) * a.nblk)), block(l.threads);
  if (c.dy)
    hipLaunchKernelGGL((gnorm_kernel<IO, V, K, UB, WIDE, true, GATE>), grid, block, 0, c.stream, a);
  else
    hipLaunchKernelGGL((gnorm_kernel<IO, V, K, UF, WIDE, false, GATE>), grid, block, 0, c.stream, a);
  return hipGetLastError();
}
template <int IO, int V, int K, int UF, int UB, bool WIDE>
hipError_t launch_typed(const GnCall& c, const Layout& l, const GnArgs& a) {
  if (a.gate == kGateNone) return launch_gate<IO, V, K, UF, UB, WIDE, kGateNone>(c, l, a);
  if (a.gate == kGateAfter) return launch_gate<IO, V, K, UF, UB, WIDE, kGateAfter>(c, l, a);
  return launch_gate<IO, V, K, UF, UB, WIDE, kGateFirst>(c, l, a);
}

template <int IO, int V>
hipError_t launch_large(const GnCall& c, const Layout& l, const GnArgs& a) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(l.tiles) * a.nblk)), block(l.threads);
  if (c.dy)
    hipLaunchKernelGGL((gnorm_large_kernel<IO, V, true>), grid, block, 0, c.stream, a);
  else
    hipLaunchKernelGGL((gnorm_large_kernel<IO, V, false>), grid, block, 0, c.stream, a);
  return hipGetLastError();
}

template <int IO>
hipError_t launch_io(const GnCall& c, const Layout& l, const GnArgs& a) {
  constexpr int V = IO == 0 ? 4 : 8;
  if (l.wide) {
    if (l.vec == 1)
      return l.k == 4 ? launch_gate<IO, 1, 4, 1, 1, true, kGateAny>(c, l, a) : launch_large<IO, 1>(c, l, a);
    return l.k == 1 ? launch_typed<IO, V, 1, 1, 1, true>(c, l, a) : launch_large<IO, V>(c, l, a);
  }
  if (l.vec == 1)
    return l.k == 2 ? launch_typed<IO, 1, 2, 1, 1, false>(c, l, a) : launch_typed<IO, 1, 8, 1, 1, false>(c, l, a);
  return launch_typed<IO, V, 1, 4, 2, false>(c, l, a);
}

}  // namespace

size_t gn_part_floats(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int sums) {
  if (sums == 0) return 0;
  // the call may take either layout, by the alignment of its tensors
  const int64_t v = blocks(layout(channels, groups, io_dtype, true, true), rows, io_dtype, true);
  const int64_t s = blocks(layout(channels, groups, io_dtype, false, true), rows, io_dtype, true);
  return static_cast<size_t>(v > s ? v : s) * channels * sums;
}

hipError_t launch_gnorm(const GnCall& c) {
  const int full = c.io_dtype == 0 ? 4 : 8;
  auto fits = [&](const void* p, int64_t row) { return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && row % full == 0; };
  const bool can_vec = fits(c.x, c.x_row) && fits(c.out, c.channels) && (!c.z || fits(c.z, c.z_row)) &&
                       (!c.dy || fits(c.dy, c.dy_row)) && (!c.dz || fits(c.dz, c.channels));
  const Layout l = layout(c.channels, c.groups, c.io_dtype, can_vec, c.dy != nullptr);
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
  a.nblk = static_cast<int32_t>(blocks(l, c.rows, c.io_dtype, c.dy != nullptr));
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
  return launch_part_sums(a.nblk, {{c.channels, a.pw, c.dweight}, {c.channels, a.pb, c.dbias}}, c.stream);
}

}  // namespace mscan
