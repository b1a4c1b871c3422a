// What the kernels that go over rows (tokens) of channels share: pieces of a
// row in one load, sums over lanes and workgroups, the activations, and the
// sum of the partial sums that workgroups leave of a parameter's gradient.
#pragma once

#include <initializer_list>

#include "mfma_frag.h"
#include "scan_device.h"

namespace mscan {

namespace {

constexpr int kActNone = 0, kActSilu = 1;  // 2: sigmoid

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
    __builtin_nontemporal_store(__builtin_bit_cast(u4, v), reinterpret_cast<u4*>(p));
  } else {
    __builtin_nontemporal_store(f4{o[0], o[1], o[2], o[3]}, reinterpret_cast<f4*>(p));
  }
}
template <int IO, int V>
__device__ __forceinline__ Vec<IO, V> fetch(const void* base, int64_t at, bool ok) {
  Vec<IO, V> r{};
  if (ok) r = *reinterpret_cast<const Vec<IO, V>*>(static_cast<const typename Io<IO>::T*>(base) + at);
  return r;
}

// V parameters of a lane's channels, `otherwise` where there are none.
template <int V>
__device__ __forceinline__ void fetch_params(const float* p, int at, bool ok, float otherwise, float (&o)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = otherwise;
  if (!p || !ok) return;
  if constexpr (V == 1) {
    o[0] = p[at];
  } else {
    typedef float f4a __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f4a v = *reinterpret_cast<const f4a*>(p + at + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i + j] = v[j];
    }
  }
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

// The same over a whole workgroup, N sums at once. Each call takes the other
// half of `red` than the call before it, so that one barrier does: who writes
// a half again has passed the barrier behind its last reading.
template <int N>
__device__ __forceinline__ void wide_sum(float (&v)[N], float (&red)[2][N][16], int half) {
  const int waves = static_cast<int>(blockDim.x) >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lanes_sum(v[i], 64);
    if ((threadIdx.x & 63) == 0) red[half][i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = red[half][i][0];
    for (int w = 1; w < waves; ++w) v[i] += red[half][i][w];
  }
}

// Values whose squares, or whose sum, leave float32 at its upper end (a sum of
// squares from 2^120 on, or NaN) are taken times 2^-80, exactly, and their
// statistics again; at its lower end (without an eps) times 2^90. Where these
// are 0 then, all values are equal, and 1 / sqrt(eps) is not scaled.
__device__ __forceinline__ float scale_for(float squares, float mean_square) {
  return !(squares < 0x1p120f) ? 0x1p-80f : mean_square < 0x1p-100f ? 0x1p90f : 1.0f;
}

// sigmoid(z) = 1 / (1 + e), e = e^-z, and 1 - sigmoid(z) = e / (1 + e), the
// latter without cancellation. Where e overflows the first is 0 and the minimum
// takes the second from infinity times 0 to 1 (a NaN is in the first).
struct Sig {
  float s, c;
};
__device__ __forceinline__ Sig sigmoid(float z) {
  const float e = exp2_hw(-z * kLog2e), s = rcp_hw(1.0f + e);
  return Sig{s, fminf(e * s, 1.0f)};
}
// z sigmoid(z). Below -128 the second factor is 0 (e^128 is beyond float32),
// and so the first may stay at -128 there: -inf closes a gate as the lowest
// value does, not as infinity times 0.
__device__ __forceinline__ float silu_of(float z, float s) { return fmaxf(z, -128.0f) * s; }
// Chosen by value, not by branch: the kind is the same for a whole launch, and
// a branch at each element would keep the elements from overlapping.
__device__ __forceinline__ float act(int kind, float z) {
  const float s = sigmoid(z).s;
  const float a = kind == kActSilu ? silu_of(z, s) : s;
  return kind == kActNone ? z : a;
}
// activation and its derivative: of silu, s + z s (1 - s)
__device__ __forceinline__ float act_grad(int kind, float z, float& a) {
  const Sig g = sigmoid(z);
  const float b = kind == kActSilu ? silu_of(z, g.s) : g.s;
  a = kind == kActNone ? z : b;
  const float d = kind == kActSilu ? fmaf(b, g.c, g.s) : g.s * g.c;
  return kind == kActNone ? 1.0f : d;
}

// out[c] = sum over blocks of part[block][c]: 16 channels a workgroup, whose 64
// quarter waves take every 64th block, four at a time.
struct PartSum {
  int32_t n;  // channels
  const float* part;
  float* out;
};
__global__ __launch_bounds__(1024) void part_sum_kernel(int32_t nblk, PartSum s0, PartSum s1, PartSum s2) {
  __shared__ float red[64][17];
  const PartSum set = blockIdx.y == 0 ? s0 : blockIdx.y == 1 ? s1 : s2;
  const float* part = set.part;
  float* out = set.out;
  const int32_t channels = set.n;
  if (!out) return;
  const int l = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + l;
  float s[4] = {};
  if (c < channels)
    for (int j = h; j < nblk; j += 256)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + 64 * k < nblk) s[k] += part[static_cast<int64_t>(j + 64 * k) * channels + c];
  red[h][l] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  // the 64 sums of a channel: 16 threads a channel, then 16 lanes together
  const int cl = threadIdx.x >> 4, hl = threadIdx.x & 15;
  if (cl < 16) {
    float t = (red[hl][cl] + red[hl + 16][cl]) + (red[hl + 32][cl] + red[hl + 48][cl]);
    t = lanes_sum(t, 16);
    if (hl == 0 && blockIdx.x * 16 + cl < channels) out[blockIdx.x * 16 + cl] = t;
  }
}

// Up to three sums of a call in one launch; a set without an output is left out.
hipError_t launch_part_sums(int32_t nblk, std::initializer_list<PartSum> sets, hipStream_t stream) {
  PartSum s[3] = {};
  int32_t n = 0, used = 0;
  for (const PartSum& set : sets)
    if (set.out) {
      n = n > set.n ? n : set.n;
      s[used++] = set;
    }
  if (!used) return hipSuccess;
  hipLaunchKernelGGL(part_sum_kernel, dim3(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>(used)), dim3(1024), 0, stream,
                     nblk, s[0], s[1], s[2]);
  return hipGetLastError();
}

}  // namespace

}  // namespace mscan
