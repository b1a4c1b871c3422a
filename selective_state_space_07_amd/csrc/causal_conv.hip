// The short causal convolution in front of a scan, depthwise over time, its
// gradients and its one-token form.
//
// Per batch row and channel, with k taps and x before the first token from the
// state:
//   u_t = b + sum_{j<k} w_j x_{t-k+1+j},   y_t = act(u_t).
// Gradients, with du_t = dy_t act'(u_t):
//   dx_s = sum_{d<k} w_{k-1-d} du_{s+d},  dw_j = sum_t du_t x_{t-k+1+j},  db = sum_t du_t.
//
// Every tensor is read and written once, so the forward is bound by memory
// traffic. A lane holds four neighbouring channels and walks a run of tokens
// with the last k - 1 inputs in registers; a wave's 64 lanes read 512 bytes of a
// bfloat16 token side by side, and a workgroup's four waves walk runs that
// follow one another. What two runs both read (k - 1 tokens) comes from the
// caches. The backward walks the same way, k - 1 tokens further: a token's dx is
// complete, and leaves, k - 1 tokens after it. u is computed again rather than
// kept. Sums over tokens stay in registers and leave as one partial sum per
// workgroup, which a second kernel adds in a fixed order.
//
// A token's number is the same in all lanes of a wave, so what depends on it
// (its run, its document) is branched on, and the branches stand where no sum
// would be copied over them: moves were a fifth of the backward's instructions.
// It takes some 27 vector instructions an element and is bound by their issue
// (76% of its time) before it is by memory. With 3 waves' registers of a SIMD
// and runs as long as it takes to give each wave one, its work is even; with
// eight channels a lane there were 2 waves, and 66 us in place of 42.
//
// Measured with four taps at 8 x 2048 tokens of 1792 channels, bfloat16: forward
// 28 us (117 MB, 4.2 TB/s); gradients 42 us (176 MB, 4.2 TB/s), and 5 us for the
// sums over workgroups; one token of 256 rows 4.9 us.
#include <algorithm>

#include "conv_internal.h"
#include "row_device.h"

namespace mscan {

namespace {

constexpr int kThreads = 256, kLn = 64, kSub = kThreads / kLn;  // lanes along a token, and runs of a workgroup

struct ConvArgs {
  int32_t batch, seqlen, channels, activation, cols, nblk, run, nruns;  // nruns: of one batch row
  int64_t runs, x_row;
  const void* x;
  const int32_t* seq_idx;
  const float *weight, *bias, *state_in, *dstate_out;
  int32_t first[kConvMaxParts];  // each part's first channel (channels behind the last part)
  void* part[kConvMaxParts];
  int64_t part_row[kConvMaxParts];
  float *state_out, *dstate_in;
  void* dx;
  float *pw, *pb;
};

// A lane's place in a part: the address of its channels in the row of token 0.
template <typename T>
struct PartAt {
  T* p;
  int64_t row;
  __device__ __forceinline__ PartAt(const ConvArgs& a, int c) {
    int i = 0;
#pragma unroll
    for (int j = 1; j < kConvMaxParts; ++j) i = c >= a.first[j] ? j : i;
    p = static_cast<T*>(a.part[i]) + (c - a.first[i]);
    row = a.part_row[i];
  }
};

// V neighbouring channels of a token, one or four, as they lie in memory: one element, or words.
template <int IO, int V>
struct Piece {
  static constexpr int kWords = IO == 1 ? V / 2 : V;
  uint32_t w[kWords];
};
template <int IO>
struct Piece<IO, 1> {
  typename Io<IO>::T v;
};
template <int IO, int V>
__device__ __forceinline__ Piece<IO, V> read(const typename Io<IO>::T* p) {
  if constexpr (V == 1) {
    return Piece<IO, 1>{*p};
  } else if constexpr (IO == 1) {
    const u2 v = *reinterpret_cast<const u2*>(p);
    return Piece<IO, V>{{v.x, v.y}};
  } else {
    const u4 v = *reinterpret_cast<const u4*>(p);
    return Piece<IO, V>{{v.x, v.y, v.z, v.w}};
  }
}
template <int IO, int V>
__device__ __forceinline__ void unpack(const Piece<IO, V>& p, float (&o)[V]) {
  if constexpr (V == 1) {
    o[0] = Io<IO>::cvt(p.v);
  } else {
#pragma unroll
    for (int i = 0; i < Piece<IO, V>::kWords; ++i) {
      if constexpr (IO == 1) {
        o[2 * i] = __uint_as_float(p.w[i] << 16);
        o[2 * i + 1] = __uint_as_float(p.w[i] & 0xFFFF0000u);
      } else {
        o[i] = __uint_as_float(p.w[i]);
      }
    }
  }
}
template <int IO, int V>
__device__ __forceinline__ void write(typename Io<IO>::T* p, const float (&o)[V]) {
  if constexpr (V == 1) {
    Io<IO>::store(p, o[0]);
  } else if constexpr (IO == 1) {
    typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
    const bf4 v = {static_cast<__bf16>(o[0]), static_cast<__bf16>(o[1]), static_cast<__bf16>(o[2]), static_cast<__bf16>(o[3])};
    *reinterpret_cast<u2*>(p) = __builtin_bit_cast(u2, v);
  } else {
    *reinterpret_cast<f4*>(p) = f4{o[0], o[1], o[2], o[3]};
  }
}

template <int V, int K>
struct Params {
  float w[K][V], b[V];
  __device__ __forceinline__ Params(const ConvArgs& a, int c) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][i] = a.weight[static_cast<int64_t>(c + i) * K + j];
      b[i] = a.bias ? a.bias[c + i] : 0.0f;
    }
  }
  // u of a token whose input is x, with the K - 1 inputs before it in `past`
  __device__ __forceinline__ void sum(const float (&past)[K - 1][V], const float (&x)[V], float (&u)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] = b[i];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) u[i] = fmaf(w[j][i], past[j][i], u[i]);
      u[i] = fmaf(w[K - 1][i], x[i], u[i]);
    }
  }
};

// The inputs before a run's first token, oldest first, and how many of them are
// of that token's document (K - 1 where the document began earlier).
template <int IO, int V, int K, bool SEQ>
struct Past {
  float x[K - 1][V];
  int age;
  __device__ __forceinline__ Past(const ConvArgs& a, const typename Io<IO>::T* row0, int b, int t0, int c) {
    age = K - 1;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = t0 - (K - 1) + j;
      if (t >= 0) {
        unpack<IO, V>(read<IO, V>(row0 + t * a.x_row), x[j]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          x[j][i] = a.state_in ? a.state_in[(static_cast<int64_t>(b) * a.channels + c + i) * (K - 1) + t + K - 1] : 0.0f;
      }
      if (SEQ) meet(t > 0 && differs(a, b, t));
      if (SEQ && age == 0)
#pragma unroll
        for (int q = 0; q < j; ++q) clear(q);
    }
  }
  static __device__ __forceinline__ bool differs(const ConvArgs& a, int b, int t) {
    const int32_t* id = a.seq_idx + static_cast<int64_t>(b) * a.seqlen + t;
    return id[0] != id[-1];
  }
  __device__ __forceinline__ void clear(int q) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[q][i] = 0.0f;
  }
  // A token comes, at which a document begins or does not.
  __device__ __forceinline__ void meet(bool begins) { age = begins ? 0 : age < K - 1 ? age + 1 : age; }
  __device__ __forceinline__ void begin(bool begins) {
    meet(begins);
#pragma unroll
    for (int q = 0; q < K - 1; ++q)
#pragma unroll
      for (int i = 0; i < V; ++i) x[q][i] = begins ? 0.0f : x[q][i];  // chosen: whatever it was
  }
  __device__ __forceinline__ void push(const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int q = 0; q < K - 2; ++q) x[q][i] = x[q + 1][i];
      x[K - 2][i] = v[i];
    }
  }
};

// The activation's derivative: of silu, s + u s (1 - s) = s (1 + u (1 - s)) with 1 - s = e^-u s, at both ends from the
// nearest u where none of these overflows or is infinity times 0 (88: off by less than 10^-36). A NaN stays one.
__device__ __forceinline__ float slope(int kind, float u) {
  u = __builtin_elementwise_minimum(__builtin_elementwise_maximum(u, -88.0f), 88.0f);
  const float e = exp2_hw(-u * kLog2e), s = rcp_hw(1.0f + e), d = s * fmaf(u, e * s, 1.0f);
  return kind == kActNone ? 1.0f : d;
}

constexpr int kU = 4;  // tokens in flight: what one held is read again, kU tokens further, once it is unpacked

template <int IO, int V, int K, bool SEQ, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(const ConvArgs a) {
  using T = typename Io<IO>::T;
  const int sub = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kLn);
  const int col = blockIdx.x % a.cols, blk = blockIdx.x / a.cols;
  const int c = (col * kLn + static_cast<int>(threadIdx.x % kLn)) * V;
  if (c >= a.channels) return;
  const Params<V, K> par(a, c);
  const PartAt<T> part(a, c);
  for (int64_t r = static_cast<int64_t>(blk) * kSub + sub; r < a.runs; r += static_cast<int64_t>(a.nblk) * kSub) {
    const int b = static_cast<int>(r / a.nruns), t0 = static_cast<int>(r - static_cast<int64_t>(b) * a.nruns) * a.run;
    const int t1 = min(t0 + a.run, a.seqlen);
    const int64_t first = static_cast<int64_t>(b) * a.seqlen;
    const T* row0 = static_cast<const T*>(a.x) + first * a.x_row + c;
    Piece<IO, V> now[kU];
    int32_t id[kU], before = 0;
    auto fetch = [&](int i, int t) {
      now[i] = read<IO, V>(row0 + min(t, t1 - 1) * a.x_row);
      if (SEQ) id[i] = a.seq_idx[first + min(t, t1 - 1)];
    };
#pragma unroll
    for (int i = 0; i < kU; ++i) fetch(i, t0 + i);
    Past<IO, V, K, SEQ> past(a, row0, b, t0, c);
    if (SEQ) before = a.seq_idx[first + max(t0 - 1, 0)];
    T* out = part.p + (first + t0) * part.row;
    for (int t = t0; t < t1; t += kU)
#pragma unroll
      for (int i = 0; i < kU; ++i) {  // behind the run's end the last token again, which does not leave
        float x[V], u[V];
        unpack<IO, V>(now[i], x);
        if (SEQ) {
          past.begin(id[i] != before);
          before = id[i];
        }
        fetch(i, t + i + kU);
        par.sum(past.x, x, u);
        past.push(x);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = SILU ? silu_of(u[e], sigmoid(u[e]).s) : u[e];
        if (t + i < t1) write<IO, V>(out, u);
        out += part.row;
      }
    if (a.state_out && t1 == a.seqlen) {
      const Past<IO, V, K, SEQ> end(a, row0, b, a.seqlen, c);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          a.state_out[(static_cast<int64_t>(b) * a.channels + c + i) * (K - 1) + j] = end.x[j][i];
    }
  }
}

template <int IO, int V, int K, bool SEQ>
__global__ __launch_bounds__(kThreads, 3) void conv_bwd_kernel(const ConvArgs a) {
  using T = typename Io<IO>::T;
  constexpr int kU = V > 1 && (IO == 0 || SEQ) ? 2 : mscan::kU;  // fewer where four would not leave three waves' registers
  __shared__ float join[kSub][kLn * V];
  const int sub = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kLn), lane = threadIdx.x % kLn;
  const int col = blockIdx.x % a.cols, blk = blockIdx.x / a.cols;
  const int c = (col * kLn + lane) * V;
  float dw[K][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][i] = 0.0f;
  }
  if (c < a.channels) {
    const Params<V, K> par(a, c);
    const PartAt<const T> part(a, c);
    for (int64_t r = static_cast<int64_t>(blk) * kSub + sub; r < a.runs; r += static_cast<int64_t>(a.nblk) * kSub) {
      const int b = static_cast<int>(r / a.nruns), t0 = static_cast<int>(r - static_cast<int64_t>(b) * a.nruns) * a.run;
      const int t1 = min(t0 + a.run, a.seqlen);  // the run's own tokens
      const int64_t first = static_cast<int64_t>(b) * a.seqlen, state0 = (static_cast<int64_t>(b) * a.channels + c) * (K - 1);
      const T* row0 = static_cast<const T*>(a.x) + first * a.x_row + c;
      const T* dy0 = part.p + first * part.row;
      T* out = static_cast<T*>(a.dx) + (first + t0) * a.channels + c;
      const int last = a.seqlen - 1;
      Piece<IO, V> now[kU], dnow[kU];
      int32_t id[kU], before = 0;
      auto fetch = [&](int i, int t) {
        now[i] = read<IO, V>(row0 + min(t, last) * a.x_row);
        dnow[i] = read<IO, V>(dy0 + min(t, last) * part.row);
        if (SEQ) id[i] = a.seq_idx[first + min(t, last)];
      };
#pragma unroll
      for (int i = 0; i < kU; ++i) fetch(i, t0 + i);
      Past<IO, V, K, SEQ> past(a, row0, b, t0, c);
      if (SEQ) before = a.seq_idx[first + max(t0 - 1, 0)];
      float acc[K][V];  // dx of the K latest tokens, oldest first
#pragma unroll
      for (int d = 0; d < K; ++d)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[d][i] = 0.0f;
      // a token's gradients, from what piece i holds; `own`: not another run's
      auto gradients = [&](int i, bool own, auto&& more) {
        float x[V], du[V], u[V];
        unpack<IO, V>(now[i], x);
        unpack<IO, V>(dnow[i], du);
        if (SEQ) {
          past.begin(id[i] != before);
          before = id[i];
        }
        more();
        par.sum(past.x, x, u);
#pragma unroll
        for (int e = 0; e < V; ++e) du[e] *= slope(a.activation, u[e]);
        if (own)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += du[e];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) dw[j][e] = fmaf(du[e], past.x[j][e], dw[j][e]);
            dw[K - 1][e] = fmaf(du[e], x[e], dw[K - 1][e]);
          }
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
          for (int d = 0; d < K; ++d) {  // the token d before this one: tap K - 1 - d met it
            const float to = acc[K - 1 - d][e];
            acc[K - 1 - d][e] = !SEQ || d <= past.age ? fmaf(par.w[K - 1 - d][e], du[e], to) : to;
          }
        past.push(x);
      };
      // dx of the token K - 1 before `at` is complete; before t0 it is another run's, or the state's
      auto leave = [&](int at) {
        if (at - (K - 1) >= t0) {
          write<IO, V>(out, acc[0]);
          out += a.channels;
        } else if (t0 == 0 && a.dstate_in) {
#pragma unroll
          for (int e = 0; e < V; ++e) a.dstate_in[state0 + e * (K - 1) + at] = acc[0][e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
          for (int d = 0; d < K - 1; ++d) acc[d][e] = acc[d + 1][e];
          acc[K - 1][e] = 0.0f;
        }
      };
      int t = t0;
      for (; t + kU <= t1; t += kU)
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          gradients(i, true, [&]() { fetch(i, t + i + kU); });
          leave(t + i);
        }
      // what is left of the run, and the K - 1 tokens behind it
#pragma unroll 1
      for (const int stop = t1 + K - 1; t < stop; ++t) {
        if (t <= last) {
          gradients(0, t < t1, []() {});
#pragma unroll
          for (int i = 0; i + 1 < kU; ++i) {
            now[i] = now[i + 1];
            dnow[i] = dnow[i + 1];
            if (SEQ) id[i] = id[i + 1];
          }
          fetch(kU - 1, t + kU);
        }
        const int in_state = t - a.seqlen;  // the token's place among the inputs that the state holds
        if (a.dstate_out && in_state >= 0 && (!SEQ || last - (t - (K - 1)) <= past.age))
#pragma unroll
          for (int e = 0; e < V; ++e) acc[0][e] += a.dstate_out[state0 + e * (K - 1) + in_state];
        leave(t);
      }
    }
  }
  // the workgroup's runs, one after the other
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    if (j == K && !a.pb) break;
#pragma unroll
    for (int i = 0; i < V; ++i) join[sub][lane * V + i] = j < K ? dw[j < K ? j : 0][i] : db[i];
    __syncthreads();
    const int e = threadIdx.x, ch = col * kLn * V + e;
    if (e < kLn * V && ch < a.channels) {
      float s = join[0][e];
#pragma unroll
      for (int q = 1; q < kSub; ++q) s += join[q][e];
      const int64_t to = static_cast<int64_t>(blk) * a.channels + ch;
      (j < K ? a.pw[to * K + j] : a.pb[to]) = s;
    }
    __syncthreads();
  }
}

// One token: a lane a channel.
template <int IO, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const ConvArgs a) {
  using T = typename Io<IO>::T;
  const int64_t n = static_cast<int64_t>(a.batch) * a.channels;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int b = static_cast<int>(i / a.channels), c = static_cast<int>(i - static_cast<int64_t>(b) * a.channels);
    const Params<1, K> par(a, c);
    const PartAt<T> part(a, c);
    float past[K - 1][1], x[1], u[1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) past[j][0] = a.state_in[i * (K - 1) + j];
    x[0] = Io<IO>::load(static_cast<const T*>(a.x) + b * a.x_row + c);
    par.sum(past, x, u);
    Io<IO>::store(part.p + b * part.row, act(a.activation, u[0]));
#pragma unroll
    for (int j = 0; j < K - 2; ++j) a.state_out[i * (K - 1) + j] = past[j + 1][0];
    a.state_out[i * (K - 1) + K - 2] = x[0];
  }
}

// Tokens of a run (a multiple of kU), runs of a batch row and workgroups that share the runs of
// `cols` column groups.
struct Split {
  int32_t run, nruns, cols, nblk;
  int64_t runs;
};
// Of the forward 32 tokens, less where that leaves workgroups too few (16: 29.8 us in place of 28.8 at 8 x 2048 tokens of
// 1792 channels); of the backward as many as give each of the three waves of every SIMD one run (32 for all: 47 us in
// place of 42).
Split split(int32_t batch, int32_t seqlen, int32_t channels, int vec, bool bwd) {
  Split s{};
  s.cols = (channels + kLn * vec - 1) / (kLn * vec);
  const int64_t slots = bwd ? 768 : int64_t{1} << 22, most = std::max<int64_t>(1, slots / s.cols);
  auto units = [&](int64_t run) {  // workgroups that all runs are, of this length
    s.run = static_cast<int32_t>(run);
    s.nruns = (seqlen + s.run - 1) / s.run;
    s.runs = static_cast<int64_t>(batch) * s.nruns;
    return (s.runs + kSub - 1) / kSub;
  };
  int64_t run = bwd ? std::max<int64_t>(kU, static_cast<int64_t>(batch) * seqlen / (most * kSub) / kU * kU) : 32, all;
  if (bwd) {
    while ((all = units(run)) > most && run < seqlen) run += std::max<int64_t>(kU, run / 16 / kU * kU);
  } else {
    while ((all = units(run)) * s.cols < 512 && run > kU) run /= 2;
  }
  const int64_t turns = (all + most - 1) / most;
  s.nblk = static_cast<int32_t>((all + turns - 1) / turns);
  return s;
}

constexpr int kVec = 4;

ConvArgs args(const ConvCall& c) {
  ConvArgs a{};
  a.batch = c.batch;
  a.seqlen = c.seqlen;
  a.channels = c.channels;
  a.activation = c.activation;
  a.x_row = c.x_row;
  a.x = c.x;
  a.seq_idx = c.seq_idx;
  a.weight = c.weight;
  a.bias = c.bias;
  a.state_in = c.state_in;
  a.dstate_out = c.dstate_out;
  a.state_out = c.state_out;
  a.dstate_in = c.dstate_in;
  a.dx = c.dx;
  int32_t first = 0;
  for (int i = 0; i < kConvMaxParts; ++i) {
    a.first[i] = i < c.parts ? first : c.channels;
    if (i >= c.parts) continue;
    a.part[i] = c.part[i];
    a.part_row[i] = c.part_row[i];
    first += c.part_channels[i];
  }
  return a;
}

bool can_vec(const ConvCall& c) {
  const size_t bytes = c.io_dtype == 0 ? sizeof(Piece<0, kVec>) : sizeof(Piece<1, kVec>);
  auto fits = [&](const void* p, int64_t row) { return reinterpret_cast<uintptr_t>(p) % bytes == 0 && row % kVec == 0; };
  bool ok = fits(c.x, c.x_row) && c.channels % kVec == 0 && (!c.dx || fits(c.dx, c.channels));
  for (int i = 0; i < c.parts; ++i) ok = ok && fits(c.part[i], c.part_row[i]) && c.part_channels[i] % kVec == 0;
  return ok;
}

template <int IO, int V, int K>
hipError_t launch_taps(const ConvCall& c, ConvArgs a) {
  const Split s = split(c.batch, c.seqlen, c.channels, V, c.dx != nullptr);
  a.cols = s.cols;
  a.nblk = s.nblk;
  a.run = s.run;
  a.nruns = s.nruns;
  a.runs = s.runs;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(s.cols) * s.nblk)), block(kThreads);
  if (!c.dx) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, c.stream, a); };
    if (c.activation == kActSilu)
      c.seq_idx ? go(conv_fwd_kernel<IO, V, K, true, true>) : go(conv_fwd_kernel<IO, V, K, false, true>);
    else
      c.seq_idx ? go(conv_fwd_kernel<IO, V, K, true, false>) : go(conv_fwd_kernel<IO, V, K, false, false>);
    return hipGetLastError();
  }
  a.pw = c.sums;
  a.pb = c.dbias ? c.sums + static_cast<size_t>(s.nblk) * c.channels * K : nullptr;
  if (c.seq_idx)
    hipLaunchKernelGGL((conv_bwd_kernel<IO, V, K, true>), grid, block, 0, c.stream, a);
  else
    hipLaunchKernelGGL((conv_bwd_kernel<IO, V, K, false>), grid, block, 0, c.stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_part_sums(s.nblk, {{c.channels * K, a.pw, c.dweight}, {c.channels, a.pb, c.dbias}}, c.stream);
}

template <int IO, int V>
hipError_t launch_vec(const ConvCall& c, const ConvArgs& a) {
  return c.taps == 2 ? launch_taps<IO, V, 2>(c, a) : c.taps == 3 ? launch_taps<IO, V, 3>(c, a) : launch_taps<IO, V, 4>(c, a);
}

template <int IO>
hipError_t launch_step_io(const ConvCall& c, const ConvArgs& a) {
  const int64_t blocks = (static_cast<int64_t>(c.batch) * c.channels + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 20))), block(kThreads);
  if (c.taps == 2)
    hipLaunchKernelGGL((conv_step_kernel<IO, 2>), grid, block, 0, c.stream, a);
  else if (c.taps == 3)
    hipLaunchKernelGGL((conv_step_kernel<IO, 3>), grid, block, 0, c.stream, a);
  else
    hipLaunchKernelGGL((conv_step_kernel<IO, 4>), grid, block, 0, c.stream, a);
  return hipGetLastError();
}

}  // namespace

size_t conv_part_floats(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps) {
  // the call may take either form, by the alignment of its tensors
  const size_t v = split(batch, seqlen, channels, kVec, true).nblk;
  const size_t s = split(batch, seqlen, channels, 1, true).nblk;
  return (v > s ? v : s) * static_cast<size_t>(channels) * (taps + 1);
}

hipError_t launch_conv(const ConvCall& c) {
  const ConvArgs a = args(c);
  const bool vec = can_vec(c);
  if (c.io_dtype == 0) return vec ? launch_vec<0, kVec>(c, a) : launch_vec<0, 1>(c, a);
  return vec ? launch_vec<1, kVec>(c, a) : launch_vec<1, 1>(c, a);
}

hipError_t launch_conv_step(const ConvCall& c) {
  const ConvArgs a = args(c);
  return c.io_dtype == 0 ? launch_step_io<0>(c, a) : launch_step_io<1>(c, a);
}

}  // namespace mscan
