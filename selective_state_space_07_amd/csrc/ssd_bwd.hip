// Gradients of the Mamba-2 SSD scan (mamba2_ssd_fwd), in chunks, on the matrix
// cores.
//
// Per batch row and head, with a_t = exp(delta_t A):
//   S_t = a_t S_{t-1} + delta_t x_t B_t^T,   y_t = S_t C_t + D x_t,
//   R_t = dy_t C_t^T + a_{t+1} R_{t+1}       (the gradient of S_t, last token first),
//   dC_t = S_t^T dy_t,  dB_t = delta_t R_t^T x_t,  dx_t = delta_t R_t B_t + D dy_t,
//   g_t = a_t <R_t, S_{t-1}> (of log a_t),  ddelta_t = x_t . R_t B_t + A g_t.
// Over a chunk of 256 tokens with cs the running sum of delta A inside it, S the
// state before it, R the gradient behind it and w_rs = exp(cs_r - cs_s), s <= r:
//   dC_r = sum_s w_rs delta_s (dy_r . x_s) B_s + exp(cs_r) S^T dy_r
//   dB_s = delta_s [ sum_r w_rs (dy_r . x_s) C_r + exp(cs_end - cs_s) R^T x_s ]
//   dx_s = delta_s [ sum_r w_rs (C_r . B_s) dy_r + exp(cs_end - cs_s) R B_s ] + D dy_s
//   g_t  = sum_{r>=t>s} m_rs + sum_{r>=t} exp(cs_r) dy_r . S C_r
//          + sum_{s<t} delta_s exp(cs_end - cs_s) x_s . R B_s + exp(cs_end) <R, S>,
//   m_rs = w_rs delta_s (dy_r . x_s) (C_r . B_s).
// The first sum of g is taken by tiles of 64 tokens: of r in t's tile with s in
// an earlier one, of s in t's tile with r in a later one, of r in a later and s
// in an earlier one, all sums of what counts alone; only inside a tile it is a
// running sum of what each token's row of m adds and its column takes away.
//
// B and C are shared by the heads of a group, so what multiplies them is summed
// over the heads first: sum_h w delta (dy . x) is kept in registers, and meets B
// and C once for all heads; C . B is made once. Kernels:
//  1. ssdb_state_kernel: each chunk's own S and R, and the running sums;
//  2. ssdb_pass_kernel: from them S before and R behind each chunk;
//  3. ssdb_carry_kernel: what they are of dC and dB, summed over the heads;
//  4. ssdb_main_kernel, a workgroup for 64 tokens of a chunk and the heads of a
//     group: four waves make dC of their 16 tokens, four dB and dx;
//  5. ssdb_step_kernel: g, ddt and the sums for dA, ddt_bias and dD.
// Running sums are float64: their differences are what is used. For bfloat16 io
// a float32 value that meets the matrix cores is two bfloat16 parts, 16 bits,
// where dB, dC and dx are made, and three where float32 outputs are. What g and
// ddelta take from inside a chunk are sums of float32 products of exact operands;
// a row and a column of m inside a tile, whose difference counts, are summed in
// float64 (in float32 dA was off by 10^-6 of itself, and by 3 10^-7 so).
//
// Steps delta A that leave nothing (large or infinite) or that are NaN: the
// running sums stay numbers, as the state kernel clamps both; what a NaN makes
// of the tokens that meet its decay is in their delta, and g's running sums start
// again at a step that leaves nothing, as at a document. That is 0.6% of the time.
//
// Measured at 8 x 2048 tokens, 24 heads in one group, d_state 128, bfloat16, 356
// us (338 to 370 by card): state 60 us (200 MB, 3.3 TB/s), pass 30, carry 78, main
// 175, step 16, sums 5. The main kernel holds 2 x 64 sums and products in registers and 142 KB of
// LDS, so two waves on a SIMD, and neither the matrix cores nor memory but what
// two waves leave of latency bounds it: 12.5 thousand clocks a head, beside 50
// thousand before and behind the heads. What was gained there: the waves that
// make dC also have R's part of dx and, of the first tile, the farthest tile's
// part of dB and dx (15 to 12.5 thousand clocks); sums pinned where they are
// made (without it they spill). The carry kernel is bound by the vector
// instructions and matrix products of two waves in turn. With the state in
// registers and the tokens in LDS it took 85 us, for its loads of single words.
#include <algorithm>
#include <type_traits>

#include "mfma_frag.h"
#include "row_device.h"
#include "ssd_bwd_internal.h"

namespace mscan {

namespace {

constexpr int kQ = 256;      // tokens of a chunk
constexpr int kTile = 64;    // tokens of a tile
constexpr int kTiles = kQ / kTile;
constexpr int kP = 64;       // headdim
constexpr int kMain = 512;   // threads of the main kernel
constexpr int kState = 256;  // threads of the state kernel

// [64] rows of W io elements (or of float32 states) in LDS. The 16-byte pieces of
// a row are exchanged by an exclusive-or with a number made of the row, so that
// 16 rows read side by side, and 8 rows of two pieces, hit every bank once.
template <int IO, int W>
struct Lds {
  using T = typename Io<IO>::T;
  static constexpr uint32_t kB = sizeof(T), kRow = W * kB, kBytes = kTile * kRow, kPer = kRow / 16;
  static __device__ __forceinline__ uint32_t exchange(uint32_t row) {
    if constexpr (kRow == 128) {
      const uint32_t u = (row >> 1) & 7;
      return (((u & 3) << 1) | (u >> 2)) << 4;
    } else {
      return (((row & 7) << 1) | ((row >> 3) & 1)) << 4;
    }
  }
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte) { return row * kRow + (byte ^ exchange(row)); }

  // 8 k-values k0 + 8 g .. of row r0 + l15 (r0 a multiple of 16, k0 of 32).
  static __device__ __forceinline__ Frag<IO> row(const char* lds, int r0, int k0, int l15, int g) {
    const uint32_t base = at(l15, 8 * kB * g);
    const char* p = lds + r0 * kRow;
    if constexpr (IO == 1) {
      return frag8(reinterpret_cast<const uint16_t*>(p + (base ^ (k0 * kB))));
    } else {
      return Frag<0>{*reinterpret_cast<const f4*>(p + (base ^ (k0 * kB))), *reinterpret_cast<const f4*>(p + (base ^ (k0 * kB + 16)))};
    }
  }
  // The same of column c + l15 (c a multiple of 16) over the rows r0 + FIRST g + j and r0 + SECOND + FIRST g + j, j < 4.
  template <int FIRST, int SECOND>
  static __device__ __forceinline__ Frag<IO> cols(const char* lds, int r0, int c, int l15, int g) {
    const char* p = lds + r0 * kRow;
    if constexpr (IO == 1) {
      // a group of 16 lanes reads 4 rows of 4 elements a lane and gets them transposed
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4* lds_s4;
      const uint32_t r = FIRST * g + (l15 >> 2), b = 2 * (4 * (l15 & 3));
      const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + (at(r, b) ^ (2 * c)))));
      const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + (at(r + SECOND, b) ^ (2 * c)))));
      const u4 v = {lo.x, lo.y, hi.x, hi.y};
      return Frag<1>{__builtin_bit_cast(bf8, v)};
    } else {
      Frag<0> f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.lo[j] = *reinterpret_cast<const float*>(p + (at(FIRST * g + j, 4 * l15) ^ (4 * c)));
        f.hi[j] = *reinterpret_cast<const float*>(p + (at(FIRST * g + SECOND + j, 4 * l15) ^ (4 * c)));
      }
      return f;
    }
  }
  // in the order of k of row(): rows r0 + 8 g ..
  static __device__ __forceinline__ Frag<IO> col(const char* lds, int r0, int c, int l15, int g) {
    return cols<8, 4>(lds, r0, c, l15, g);
  }
  // in the order in which two tiles of accumulators are an operand
  static __device__ __forceinline__ Frag<IO> col_acc(const char* lds, int r0, int c, int l15, int g) {
    return cols<4, 16>(lds, r0, c, l15, g);
  }
  // four neighbouring elements c .. of a row (c a multiple of 4)
  static __device__ __forceinline__ f4 four(const char* lds, int row, int c) {
    const char* p = lds + at(row, c * kB);
    if constexpr (IO == 1) {
      const u2 v = *reinterpret_cast<const u2*>(p);
      return f4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                __uint_as_float(v.y & 0xFFFF0000u)};
    } else {
      return *reinterpret_cast<const f4*>(p);
    }
  }
  // rows [first, last) of 64 from memory, 0 for the others
  template <int NT>
  struct Way {
    static constexpr int kN = kTile * kPer / NT;
    u4 v[kN];
    __device__ __forceinline__ void load(const T* src, int64_t ld, int first, int last, int tid) {
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        const int i = tid + q * NT, r = i / kPer, c = i % kPer;
        v[q] = u4{0, 0, 0, 0};
        if (r >= first && r < last) v[q] = *reinterpret_cast<const u4*>(src + r * ld + c * (16 / kB));
      }
    }
    __device__ __forceinline__ void store(char* lds, int tid) const {
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        const int i = tid + q * NT;
        *reinterpret_cast<u4*>(lds + at(i / kPer, i % kPer * 16)) = v[q];
      }
    }
  };
  template <int NT>
  static __device__ __forceinline__ void fill(char* lds, const T* src, int64_t ld, int first, int last, int tid) {
    Way<NT> way;
    way.load(src, ld, first, last, tid);
    way.store(lds, tid);
  }
};

// A float32 operand: for bfloat16 io as NP bfloat16 parts, the largest first. The first of three is cut, not rounded.
template <int IO, int NP>
struct Wide {
  Frag<IO> p[IO == 1 ? NP : 1];
};
__device__ __forceinline__ uint32_t round2(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
// Two values' parts as words of two bfloat16.
template <int NP>
__device__ __forceinline__ void parts2(float a, float b, uint32_t (&w)[NP]) {
#pragma clang fp contract(off)  // the parts are of the rounded values, whatever made these
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    w[p] = p == 0 && NP == 3 ? __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u) : round2(a, b);
    a -= __uint_as_float(w[p] << 16);
    b -= __uint_as_float(w[p] & 0xFFFF0000u);
  }
}
template <int IO, int NP>
__device__ __forceinline__ Wide<IO, NP> wide(f4 a, f4 b) {
  Wide<IO, NP> o;
  if constexpr (IO == 1) {
    uint32_t w[4][NP];
    parts2<NP>(a.x, a.y, w[0]);
    parts2<NP>(a.z, a.w, w[1]);
    parts2<NP>(b.x, b.y, w[2]);
    parts2<NP>(b.z, b.w, w[3]);
#pragma unroll
    for (int p = 0; p < NP; ++p) o.p[p] = Frag<1>{__builtin_bit_cast(bf8, u4{w[0][p], w[1][p], w[2][p], w[3][p]})};
  } else {
    o.p[0] = Frag<0>{a, b};
  }
  return o;
}
template <int IO, int NP>
__device__ __forceinline__ f4 mma_wide(const Frag<IO>& a, const Wide<IO, NP>& b, f4 c) {
#pragma unroll
  for (int p = (IO == 1 ? NP : 1) - 1; p >= 0; --p) c = mma(a, b.p[p], c);
  return c;
}
template <int IO, int NP>
__device__ __forceinline__ f4 mma_wide(const Wide<IO, NP>& a, const Frag<IO>& b, f4 c) {
#pragma unroll
  for (int p = (IO == 1 ? NP : 1) - 1; p >= 0; --p) c = mma(a.p[p], b, c);
  return c;
}

// A state [64][N] float32 in LDS: for bfloat16 io its NP parts, one after the other.
template <int IO, int N, int NP>
struct LdsState {
  using L = Lds<IO, N>;
  static constexpr int kParts = IO == 1 ? NP : 1;
  static constexpr uint32_t kBytes = kParts * L::kBytes;
  static __device__ __forceinline__ Wide<IO, NP> row(const char* lds, int r0, int k0, int l15, int g) {
    Wide<IO, NP> o;
#pragma unroll
    for (int p = 0; p < kParts; ++p) o.p[p] = L::row(lds + p * L::kBytes, r0, k0, l15, g);
    return o;
  }
  static __device__ __forceinline__ Wide<IO, NP> col(const char* lds, int r0, int c, int l15, int g) {
    Wide<IO, NP> o;
#pragma unroll
    for (int p = 0; p < kParts; ++p) o.p[p] = L::col(lds + p * L::kBytes, r0, c, l15, g);
    return o;
  }
};
// Its way there from memory: a thread takes four neighbouring elements at a time.
template <int IO, int N, int NT>
struct StateWay {
  static constexpr int kN = kP * N / 4 / NT;
  f4 v[kN];
  __device__ __forceinline__ void load(const float* src, int tid) {
#pragma unroll
    for (int q = 0; q < kN; ++q) v[q] = reinterpret_cast<const f4*>(src)[tid + q * NT];
  }
  template <int NP>
  __device__ __forceinline__ void store(char* lds, int tid) const {
    using L = Lds<IO, N>;
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const uint32_t i = tid + q * NT;
      char* to = lds + L::at(i / (N / 4), i % (N / 4) * 4 * L::kB);
      if constexpr (IO == 1) {
        uint32_t lo[NP], hi[NP];
        parts2<NP>(v[q].x, v[q].y, lo);
        parts2<NP>(v[q].z, v[q].w, hi);
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<u2*>(to + p * L::kBytes) = u2{lo[p], hi[p]};
      } else {
        *reinterpret_cast<f4*>(to) = v[q];
      }
    }
  }
  // what store<NP> put there of v[q]
  template <int NP>
  static __device__ __forceinline__ f4 back(const char* lds, int q, int tid) {
    using L = Lds<IO, N>;
    const uint32_t i = tid + q * NT;
    const char* from = lds + L::at(i / (N / 4), i % (N / 4) * 4 * L::kB);
    f4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (IO == 1) {
#pragma unroll
      for (int p = NP - 1; p >= 0; --p) {
        const u2 w = *reinterpret_cast<const u2*>(from + p * L::kBytes);
        o += f4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
      }
    } else {
      o = *reinterpret_cast<const f4*>(from);
    }
    return o;
  }
};

struct SbArgs {
  int32_t batch, seqlen, nheads, ngroups, d_state, nchunks;
  int32_t hsplit, per, csplit, cper;  // workgroups that share a group's heads, and the heads of one: main and carry kernel
  int64_t x_row, dt_row, b_row, c_row, dy_row;
  const void *x, *dt, *B, *C, *dy;
  const int32_t* seq_idx;
  const float *dt_bias, *A, *D, *state_in, *dstate_out;
  void *dx, *ddt, *dB, *dC;
  float *ddt_bias, *dA, *dD, *dstate_in;
  // workspace; "bch" numbers (batch row, chunk, head)
  float *S, *R;        // [bch][64][N]
  float* decay;        // [bch]: over the chunk, -1 where a document begins in it
  double* cs;          // [bch][256]
  float* delta;        // [bch][256]; its sign is set where a step behind the token, of its document and chunk, is NaN
  int32_t *begin, *next;  // [batch][chunk][256]: the latest document begin up to a token (-1: none), the first behind it (256)
  float* dot;          // [bch][16]: shares of <R, S>
  float* tok;          // [kTokSums][bch][256]
  int64_t tok_step;
  float *dBp, *dCp;    // [hsplit][batch][seqlen][ngroups][N], where hsplit > 1
  float *dBc, *dCc;    // [csplit][batch][seqlen][ngroups][N]: what the states carry
  float *pA, *pb, *pD; // [batch][chunk][heads]
};
// What the step kernel has of each token: its row of m inside its tile (before the token; in two floats, as its column) and over the three tiles before
// it, nearest first; its column inside its tile and over the tiles behind it; its shares in g of S and, without delta, of
// R, whether or not these reach it; x . dx without delta and D, but for R's share; dy . x. In float32 but for what is inside a
// tile: the others are sums that count as they are, not their differences, and off by their own float32 sums already.
enum { kRowIn, kRow1, kRow2, kRow3, kColIn, kColOut, kOfS, kOfR, kDirect, kSkip, kRowInLess, kColInLess, kTokSums };

// Steps of the exponent. Nothing is left of float32 behind one of kGone or less (2^-150 and less); one below kLeast, -infinity
// among them, counts as kLeast: it leaves as little, and the sums behind it keep the bits that their differences need.
// One that is NaN counts as kLeast too, so that the differences behind it are numbers; its delta is NaN, which is in all that
// the tokens from it on have of it, and the tokens before it, which meet its decay, have NaN for a delta of their own.
constexpr double kGone = -104.0, kLeast = -512.0;
__device__ __forceinline__ float own_delta(float d) { return __float_as_int(d) < 0 ? __builtin_nanf("") : d; }
// exp of a difference of running sums, at most 0
__device__ __forceinline__ float decayed(double d) { return exp2_hw(fminf(static_cast<float>(d) * kLog2e, 0.0f)); }

// Inclusive scan over the 256 threads of a workgroup, f(earlier, later).
template <typename V, typename F>
__device__ __forceinline__ V scan256(V v, V* part, int tid, F f) {
  const int lane = tid & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V u = __shfl_up(v, o, 64);
    if (lane >= o) v = f(u, v);
  }
  if (lane == 63) part[tid >> 6] = v;
  __syncthreads();
  for (int w = (tid >> 6) - 1; w >= 0; --w) v = f(part[w], v);
  return v;
}

// A running sum over the threads that starts again where `restart` is; without one, of scan256's bits.
__device__ __forceinline__ double scan256_runs(double v, bool restart, double* part, int* ipart, int tid) {
  const int lane = tid & 63;
  int cut = restart;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double u = __shfl_up(v, o, 64);
    const int c = __shfl_up(cut, o, 64);
    if (lane >= o) {
      if (!cut) v = u + v;
      cut |= c;
    }
  }
  if (lane == 63) {
    part[tid >> 6] = v;
    ipart[tid >> 6] = cut;
  }
  __syncthreads();
  for (int w = (tid >> 6) - 1; w >= 0 && !cut; --w) {
    v = part[w] + v;
    cut = ipart[w];
  }
  return v;
}

// 1. One chunk's own S (which 0), or R (1): w_s delta_s x_s B_s^T or w_r dy_r C_r^T summed over the tokens that reach its
// end (its beginning). A wave has 16 columns of x.
template <int IO, int N, bool SEQ>
__global__ __launch_bounds__(kState) void ssdb_state_kernel(const SbArgs a) {
  using T = typename Io<IO>::T;
  using LB = Lds<IO, N>;
  using LX = Lds<IO, kP>;
  __shared__ __attribute__((aligned(512))) char bs[LB::kBytes];
  __shared__ __attribute__((aligned(512))) char xs[LX::kBytes];
  __shared__ __attribute__((aligned(16))) float w[kQ];
  __shared__ double part[4], cs_end;
  __shared__ int ipart[4], ends[2];
  __shared__ uint8_t marks[kQ];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, l15 = lane & 15, g = lane >> 4;
  const int which = blockIdx.x & 1, c = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z;
  const int grp = h / (a.nheads / a.ngroups);
  const int valid = min(kQ, a.seqlen - c * kQ);
  const int64_t row0 = static_cast<int64_t>(b) * a.seqlen + static_cast<int64_t>(c) * kQ;
  const int64_t bc = static_cast<int64_t>(b) * a.nchunks + c, bch = bc * a.nheads + h;

  float delta = 0.0f;
  if (tid < valid) delta = softplus(Io<IO>::load(static_cast<const T*>(a.dt) + (row0 + tid) * a.dt_row + h) + a.dt_bias[h]);
  // the running sum; a document's begin starts it again, so that what another holds is no part of it
  bool restart = false;
  if (SEQ) restart = tid < valid && static_cast<int64_t>(c) * kQ + tid > 0 && a.seq_idx[row0 + tid] != a.seq_idx[row0 + tid - 1];
  double own = tid < valid ? static_cast<double>(delta) * a.A[h] : 0.0;
  const bool lost = !(own < INFINITY);
  if (lost) delta = __builtin_nanf("");
  own = lost || own < kLeast ? kLeast : own;
  asm volatile("" : "+v"(own));  // rounded here, and not with the first sum
  const double cs = SEQ ? scan256_runs(own, restart, part, ipart, tid) : scan256(own, part, tid, [](double p, double q) { return p + q; });
  if (SEQ) __syncthreads();
  if (tid == kQ - 1) cs_end = cs;
  int first = 0, last = valid;  // the tokens that count
  if (SEQ) {
    const int begin = scan256(restart ? tid : -1, ipart, tid, [](int p, int q) { return p > q ? p : q; });
    __syncthreads();
    // the first begin behind a token: a scan from the last one
    const bool mirror = kQ - 1 - tid < valid && static_cast<int64_t>(c) * kQ + kQ - 1 - tid > 0 &&
                        a.seq_idx[row0 + kQ - 1 - tid] != a.seq_idx[row0 + kQ - 2 - tid];
    const int at = scan256(mirror ? kQ - 1 - tid : kQ, ipart, tid, [](int p, int q) { return p < q ? p : q; });
    if (tid == kQ - 1) {
      ends[0] = max(begin, 0);
      ends[1] = min(at, valid);
    }
    if (h == 0 && which == 0) {
      a.begin[bc * kQ + tid] = begin;
      if (kQ - 1 - tid > 0) a.next[bc * kQ + kQ - 2 - tid] = at;
      if (tid == 0) a.next[bc * kQ + kQ - 1] = kQ;
    }
  }
  bool tainted = false, behind = false;  // a step behind the token, of its document, is NaN; one up to it, from the chunk's first on
  const bool any_lost = __syncthreads_or(lost);
  if (any_lost) {
    marks[tid] = static_cast<uint8_t>(lost | restart << 1);
    __syncthreads();
    for (int t = tid + 1; t < valid && !(marks[t] & 2); ++t) tainted |= marks[t] & 1;
    for (int t = 0; t <= tid; ++t) behind |= marks[t] & 1;
  }
  const bool open = !SEQ || (ends[1] == valid && ends[0] == 0);  // no document begins behind the chunk's first token
  if (SEQ) {
    if (which == 0) first = ends[0];
    else last = ends[1];
  }
  if (which == 0) {
    a.cs[bch * kQ + tid] = cs;
    a.delta[bch * kQ + tid] = __builtin_copysignf(delta, tainted ? -1.0f : 1.0f);
    // (a begin at the first token leaves ends[0] at 0 as well, and ends[1] too)
    if (tid == 0) a.decay[bch] = !open ? -1.0f : any_lost ? __builtin_nanf("") : decayed(cs_end);
  }
  w[tid] = tid < first || tid >= last ? 0.0f : which == 0 ? decayed(cs_end - cs) * delta : behind ? __builtin_nanf("") : decayed(cs);
  const T* X = (which == 0 ? static_cast<const T*>(a.x) + row0 * a.x_row : static_cast<const T*>(a.dy) + row0 * a.dy_row) + h * kP;
  const T* Bc = (which == 0 ? static_cast<const T*>(a.B) + row0 * a.b_row : static_cast<const T*>(a.C) + row0 * a.c_row) + grp * N;
  const int64_t ldx = which == 0 ? a.x_row : a.dy_row, ldb = which == 0 ? a.b_row : a.c_row;

  f4 acc[N / 16];
#pragma unroll
  for (int nt = 0; nt < N / 16; ++nt) acc[nt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  // tokens that do not count are 0 in both: what they hold may be infinite
  typename LB::template Way<kState> wayb;
  typename LX::template Way<kState> wayx;
  auto fetch = [&](int s0) {
    wayb.load(Bc + s0 * ldb, ldb, first - s0, last - s0, tid);
    wayx.load(X + s0 * ldx, ldx, first - s0, last - s0, tid);
  };
  int s0 = first / kTile * kTile;
  if (s0 < last) fetch(s0);
  for (; s0 < last; s0 += kTile) {
    __syncthreads();
    wayb.store(bs, tid);
    wayx.store(xs, tid);
    __syncthreads();
    if (s0 + kTile < last) fetch(s0 + kTile);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const Frag<IO> xf = LX::col(xs, 32 * kb, 16 * wv, l15, g);
      const f4 w0 = *reinterpret_cast<const f4*>(w + s0 + 32 * kb + 8 * g), w1 = *reinterpret_cast<const f4*>(w + s0 + 32 * kb + 8 * g + 4);
      f4 lo, hi;
      if constexpr (IO == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = static_cast<float>(xf.v[j]) * w0[j];
          hi[j] = static_cast<float>(xf.v[4 + j]) * w1[j];
        }
      } else {
        lo = xf.lo * w0;
        hi = xf.hi * w1;
      }
      const Wide<IO, 3> v = wide<IO, 3>(lo, hi);
#pragma unroll
      for (int nt = 0; nt < N / 16; ++nt) acc[nt] = mma_wide(LB::col(bs, 32 * kb, 16 * nt, l15, g), v, acc[nt]);
    }
  }
  // rows n = 16 nt + 4 g + j, column p = 16 wv + l15
  float* out = (which == 0 ? a.S : a.R) + bch * (kP * N) + (16 * wv + l15) * N;
#pragma unroll
  for (int nt = 0; nt < N / 16; ++nt) *reinterpret_cast<f4*>(out + 16 * nt + 4 * g) = acc[nt];
}

// 2. S before each chunk (which 0, the first chunk first), R behind it (1, the last first), in place of the chunks' own. A
// thread carries 4 neighbouring elements.
__global__ __launch_bounds__(kState) void ssdb_pass_kernel(const SbArgs a, int n4) {
  const int e = static_cast<int>(blockIdx.x >> 1) * kState + static_cast<int>(threadIdx.x), which = blockIdx.x & 1;
  if (e >= n4) return;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.nheads + h;
  const float* from = which == 0 ? a.state_in : a.dstate_out;
  f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (from) s = reinterpret_cast<const f4*>(from)[bh * n4 + e];
  f4* all = reinterpret_cast<f4*>(which == 0 ? a.S : a.R);
  constexpr int kAhead = 8;  // chunks in flight
  const int n = a.nchunks;
  f4 own[kAhead];
  float d[kAhead];
  auto slot = [&](int i) {
    const int c = which == 0 ? i : n - 1 - i;
    return (static_cast<int64_t>(b) * n + c) * a.nheads + h;
  };
  for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = slot(min(i0 + i, n - 1));
      own[i] = all[at * n4 + e];
      d[i] = a.decay[at];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= n) break;
      all[slot(i0 + i) * n4 + e] = s;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // past a document's begin nothing is carried, whatever it was; past a decay of 0 what is not finite
        s[j] = d[i] < 0.0f ? own[i][j] : fmaf(d[i], s[j], own[i][j]);
    }
  }
  if (which == 1 && a.dstate_in) reinterpret_cast<f4*>(a.dstate_in)[bh * n4 + e] = s;
}

// Sum over the four lanes that hold one token's features, in all of them.
__device__ __forceinline__ float over_g(float v) {
  uint32_t u = __float_as_uint(v);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  u = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ double over_g(double v) {
#pragma unroll
  for (int step = 0; step < 2; ++step) {
    const uint32_t lo = static_cast<uint32_t>(__double2loint(v)), hi = static_cast<uint32_t>(__double2hiint(v));
    const auto l = step == 0 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false) : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto u = step == 0 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false) : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    v = __hiloint2double(static_cast<int>(u[0]), static_cast<int>(l[0])) + __hiloint2double(static_cast<int>(u[1]), static_cast<int>(l[1]));
  }
  return v;
}

// 3. What the states are of dC (from S and dy) or of dB (from R and x), a chunk's 256 tokens at a time, with each token's
// share in g, C_r . exp(cs_r) S^T dy_r or (without delta) B_s . exp(cs_end - cs_s) R^T x_s, and that of <R, S>. A wave has
// 32 tokens, each a lane's column. What a head needs from memory is fetched while the head before it is multiplied.
template <int IO, int N>
struct CarryLds {
  static constexpr int kTok = IO == 1 ? 2 : 1;                     // tokens of a lane
  static constexpr int kRows = 128 * kTok;                         // of a workgroup
  static constexpr int kPad = 16;                                  // bytes behind a row of C (B)
  static constexpr uint32_t kRow = N * sizeof(typename Io<IO>::T) + kPad, kState = LdsState<IO, N, 3>::kBytes;
  static constexpr uint32_t kBytes = kState + kRows * kRow;
};
template <int IO, int N, bool SEQ, bool OF_C>
__device__ __forceinline__ void ssdb_carry(const SbArgs& a, int u, char* lds) {
  using T = typename Io<IO>::T;
  using CL = CarryLds<IO, N>;
  constexpr int kNt = N / 16, kTok = CL::kTok, kParts = kQ / CL::kRows;
  using LS = LdsState<IO, N, 3>;
  using Way = StateWay<IO, N, kMain>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l15 = lane & 15, g = lane >> 4;
  const int from = u % kParts * CL::kRows;
  u /= kParts;
  const int hs = u % a.csplit;
  u /= a.csplit;
  const int grp = u % a.ngroups;
  u /= a.ngroups;
  const int c = u % a.nchunks, b = u / a.nchunks;
  const int valid = min(kQ, a.seqlen - c * kQ), rep = a.nheads / a.ngroups;
  if (b >= a.batch) return;   // the grid is rounded up
  if (from >= valid) return;  // the whole workgroup; its tokens' shares are read by none
  const int h0 = grp * rep + hs * a.cper, h1 = min(h0 + a.cper, (grp + 1) * rep);
  const int64_t row0 = static_cast<int64_t>(b) * a.seqlen + static_cast<int64_t>(c) * kQ;
  const int64_t bc = static_cast<int64_t>(b) * a.nchunks + c;
  const float* const states = OF_C ? a.S : a.R;
  const int64_t ld = OF_C ? a.dy_row : a.x_row;
  int at[kTok];
  bool open[kTok];
  const T* tp[kTok];  // the tokens' rows of dy (x)
  char* const rows = lds + CL::kState;
  {  // and of C (B), in LDS
    const T* base = static_cast<const T*>(OF_C ? a.C : a.B) + grp * N;
    const int64_t ldb = OF_C ? a.c_row : a.b_row;
    constexpr int kPer = N * sizeof(T) / 8;
    for (int i = tid; i < CL::kRows * kPer; i += kMain) {
      const int r = i / kPer, o = i % kPer, t = from + r;
      const T* row = base + (row0 + (t < valid ? t : 0)) * ldb;
      *reinterpret_cast<u2*>(rows + r * CL::kRow + o * 8) = *reinterpret_cast<const u2*>(row + o * (8 / sizeof(T)));
    }
  }
  float sum[kTok][kNt][4];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    at[k] = from + 16 * kTok * wave + 16 * k + l15;
    open[k] = at[k] < valid;
    const int64_t row = row0 + (at[k] < valid ? at[k] : 0);
    if (SEQ) open[k] = open[k] && (OF_C ? a.begin[bc * kQ + at[k]] < 0 : a.next[bc * kQ + at[k]] >= kQ);
    tp[k] = static_cast<const T*>(OF_C ? a.dy : a.x) + row * ld + 8 * g;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[k][nt][j] = 0.0f;
  }
  Way way;
  Frag<IO> f[kTok][2];
  double cs[kTok], end = 0.0;
  float delta[kTok] = {};
  auto fetch = [&](int h) {
    const int64_t bch = bc * a.nheads + h;
    way.load(states + bch * (kP * N), tid);
    if (!OF_C) end = a.cs[bch * kQ + kQ - 1];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) f[k][kb] = frag8(tp[k] + h * kP + 32 * kb);
      cs[k] = a.cs[bch * kQ + at[k]];
      if (!OF_C) delta[k] = a.delta[bch * kQ + at[k]];
    }
  };
  fetch(h0);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const int64_t bch = bc * a.nheads + h;
    __syncthreads();  // the last head's state has been read
    way.template store<3>(lds, tid);
    // half of <R, S> is of either state's workgroup; what it takes of the other state comes before the next head's
    constexpr int kDot = Way::kN / 2;
    f4 other[kDot];
    if (from == 0) {
      const f4* src = reinterpret_cast<const f4*>((OF_C ? a.R : a.S) + bch * (kP * N)) + tid + (OF_C ? 0 : kDot * kMain);
#pragma unroll
      for (int q = 0; q < kDot; ++q) other[q] = src[q * kMain];
    }
    Frag<IO> now[kTok][2];
    float e[kTok], de[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) now[k][kb] = f[k][kb];
      e[k] = decayed(OF_C ? cs[k] : end - cs[k]);
      de[k] = OF_C ? e[k] : own_delta(delta[k]) * e[k];
    }
    __syncthreads();
    fetch(h + 1 < h1 ? h + 1 : h);
    float share[kTok] = {};
    int l = l15, gg = g;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      asm volatile("" : "+v"(l), "+v"(gg));  // places worked out anew: kept, they would cost the sums' registers
      f4 v[kTok];
#pragma unroll
      for (int k = 0; k < kTok; ++k) v[k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const Wide<IO, 3> sf = LS::col(lds, 32 * kb, 16 * nt, l, gg);
#pragma unroll
        for (int k = 0; k < kTok; ++k) v[k] = mma_wide(sf, now[k][kb], v[k]);
      }
#pragma unroll
      for (int k = 0; k < kTok; ++k) {
        const char* own = rows + (16 * kTok * wave + 16 * k + l) * CL::kRow + (16 * nt + 4 * gg) * sizeof(T);
        float with[4];
        if constexpr (IO == 1) {
          const u2 o = *reinterpret_cast<const u2*>(own);
          with[0] = __uint_as_float(o.x << 16);
          with[1] = __uint_as_float(o.x & 0xFFFF0000u);
          with[2] = __uint_as_float(o.y << 16);
          with[3] = __uint_as_float(o.y & 0xFFFF0000u);
        } else {
          const u2 p = reinterpret_cast<const u2*>(own)[0], q = reinterpret_cast<const u2*>(own)[1];
          with[0] = __uint_as_float(p.x);
          with[1] = __uint_as_float(p.y);
          with[2] = __uint_as_float(q.x);
          with[3] = __uint_as_float(q.y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[k][nt][j] = fmaf(v[k][j], de[k], sum[k][nt][j]);
          share[k] = fmaf(v[k][j], with[j], share[k]);
        }
      }
    }
    // a token that the state does not reach has sums of its own too: of these none counts
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      share[k] = over_g(share[k]) * e[k];
      if (g == 0) a.tok[(OF_C ? kOfS : kOfR) * a.tok_step + bch * kQ + at[k]] = share[k];
    }
    if (from == 0) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kDot; ++q) {
        const f4 own = Way::template back<3>(lds, OF_C ? q : kDot + q, tid);
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(own[j], other[q][j], s);
      }
      s = lanes_sum(s, 64);
      if (lane == 0) a.dot[bch * 16 + (OF_C ? 0 : 8) + wave] = s;
    }
  }
  float* out = (OF_C ? a.dCc : a.dBc) + hs * (static_cast<int64_t>(a.batch) * a.seqlen * a.ngroups * N);
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    if (at[k] >= valid) continue;
    float* to = out + ((row0 + at[k]) * a.ngroups + grp) * N + 4 * g;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      f4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = open[k] ? sum[k][nt][j] : 0.0f;
      *reinterpret_cast<f4*>(to + 16 * nt) = v;
    }
  }
}
template <int IO, int N, bool SEQ>
__global__ __launch_bounds__(kMain) void ssdb_carry_kernel(const SbArgs a) {
  __shared__ __attribute__((aligned(512))) char lds[CarryLds<IO, N>::kBytes];
  const int id = blockIdx.y * gridDim.x + blockIdx.x, u = id >> 1;
  if (id & 1)
    ssdb_carry<IO, N, SEQ, false>(a, u, lds);
  else
    ssdb_carry<IO, N, SEQ, true>(a, u, lds);
}

// What lies in LDS for a head of the main kernel: x of the tiles up to the own one and dy of those from it on; R; tables:
// decays to the end of a token's tile, with delta, and from the end of the tile before it, delta, and the running sums; and
// what the waves that make dC have of dx. For bfloat16 io all but R and the latter twice: one head's is filled while the
// other's is read.
struct MainTables {
  double cs[kQ];
  float to_end[kQ], from_end[kQ], delta[kQ];
  float D, unused[3];
};
template <int IO, int N>
struct MainLds {
  static constexpr int kBufs = IO == 1 ? 2 : 1, kSlots = kTiles + 1;
  static constexpr uint32_t kX = Lds<IO, kP>::kBytes, kState = LdsState<IO, N, 2>::kBytes;
  static constexpr uint32_t kR = kBufs * kSlots * kX, kDx = kR + kState, kCol = kDx + kTile * kP * 4, kTab = kCol + 256 * 4,
                            kBytes = kTab + kBufs * static_cast<uint32_t>(sizeof(MainTables));
  // before and behind the heads, B and C of a tile stand in the places of these; behind them, what the waves that make dC
  // have of dB
  static constexpr uint32_t kB = kR, kC = 0, kDB = 0;
  static_assert(Lds<IO, N>::kBytes <= kR && Lds<IO, N>::kBytes <= kState && kTile * N * 4 <= kR && kBytes <= 160 * 1024, "LDS");
};
struct MainPlace {
  int i, ntiles, valid, h0, h1, hs, grp, b, c;
};

// What fills a head's LDS: NT threads.
template <int IO, int N, int NT>
struct MainFill {
  using T = typename Io<IO>::T;
  using LX = Lds<IO, kP>;
  using M = MainLds<IO, N>;
  static constexpr int kN = kTile * LX::kPer / NT, kStep = kQ / (NT < kQ ? NT : kQ);
  static_assert(NT >= kQ, "a thread a token");
  u4 v[M::kSlots][kN];
  StateWay<IO, N, NT> r;
  double cs, end, start;
  float delta, D;

  __device__ __forceinline__ void load(const SbArgs& a, const MainPlace& pl, int h, int tid) {
    const int64_t row0 = static_cast<int64_t>(pl.b) * a.seqlen + static_cast<int64_t>(pl.c) * kQ;
    const int64_t bch = (static_cast<int64_t>(pl.b) * a.nchunks + pl.c) * a.nheads + h;
#pragma unroll
    for (int slot = 0; slot < M::kSlots; ++slot) {
      const bool is_x = slot <= pl.i;
      const int tile = is_x ? slot : slot - 1, most = max(pl.valid - 1 - tile * kTile, 0);
      const int64_t ld = is_x ? a.x_row : a.dy_row;
      const T* src = static_cast<const T*>(is_x ? a.x : a.dy) + (row0 + min(tile * kTile, pl.valid - 1)) * ld + h * kP;
#pragma unroll
      for (int q = 0; q < kN; ++q) {  // rows behind the last repeat it: no branch around a load
        const int i = tid + q * NT;
        v[slot][q] = *reinterpret_cast<const u4*>(src + min(i / static_cast<int>(LX::kPer), most) * ld + i % LX::kPer * (16 / LX::kB));
      }
    }
    r.load(a.R + bch * (kP * N), tid);
    if (tid < kQ) {
      const double* all = a.cs + bch * kQ;
      cs = all[tid];
      end = all[tid | (kTile - 1)];
      start = tid >= kTile ? all[(tid & -kTile) - 1] : 0.0;
      delta = a.delta[bch * kQ + tid];
    }
    D = a.D[h];
  }
  __device__ __forceinline__ void store(const MainPlace& pl, char* lds, int buf, int tid) const {
    const bool whole = pl.valid == kQ;
#pragma unroll
    for (int slot = 0; slot < M::kSlots; ++slot)
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        const int i = tid + q * NT, row = i / LX::kPer;
        u4 o = v[slot][q];
        if (!whole && (slot <= pl.i ? slot : slot - 1) * kTile + row >= pl.valid) o = u4{0, 0, 0, 0};
        *reinterpret_cast<u4*>(lds + (buf * M::kSlots + slot) * M::kX + LX::at(row, i % LX::kPer * 16)) = o;
      }
    r.template store<2>(lds + M::kR, tid);
    if (tid < kQ) {
      MainTables& tab = reinterpret_cast<MainTables*>(lds + M::kTab)[buf];
      tab.cs[tid] = cs;
      tab.delta[tid] = delta;
      tab.to_end[tid] = decayed(end - cs) * fabsf(delta);
      tab.from_end[tid] = decayed(cs - start);
      if (tid == 0) tab.D = D;
    }
  }
};

// One task of the main kernel: dC of 16 tokens (MAKES_C), or dB and dx of them, which meet FAR tiles beside their own. The
// other waves do the other task; they meet at the same barriers. The former also have what R has of dx, which the latter
// take over at the second barrier of a head. With HELP, of the first of four tiles, which the two meet one and four
// others of, they have the farthest tile's part of dB and dx too. The task with registers left fetches the next head for
// both (LOADS). A token is a lane's column throughout.
template <int IO, int N, bool SEQ, bool MAKES_C, int FAR, bool LOADS, bool HELP>
__device__ __forceinline__ void ssdb_task(const SbArgs& a, const MainPlace& pl, char* lds) {
  using T = typename Io<IO>::T;
  using LX = Lds<IO, kP>;
  using LB = Lds<IO, N>;
  using LS = LdsState<IO, N, 2>;
  using M = MainLds<IO, N>;
  constexpr int kNt = N / 16, kNb = N / 32, kHalf = kMain / 2, kLast = kTiles - 1;
  constexpr bool kHelps = HELP && MAKES_C;
  const int tid = threadIdx.x, lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const int i = pl.i, ntiles = pl.ntiles, valid = pl.valid;
  const int64_t row0 = static_cast<int64_t>(pl.b) * a.seqlen + static_cast<int64_t>(pl.c) * kQ;
  const int64_t bc = static_cast<int64_t>(pl.b) * a.nchunks + pl.c;
  const T* Bg = static_cast<const T*>(a.B) + row0 * a.b_row + pl.grp * N;
  const T* Cg = static_cast<const T*>(a.C) + row0 * a.c_row + pl.grp * N;
  const int own = i * kTile + 16 * w + l15;  // the lane's token in the chunk
  const bool live = own < valid;
  int begin = 0, next = kQ;  // the tokens that it meets begin, and end, here
  if (SEQ) {
    begin = a.begin[bc * kQ + own];
    next = a.next[bc * kQ + own];
  }
  auto rows_in = [&](int k) { return min(kTile, valid - k * kTile); };
  // a place in a loop from which on what follows from the lane's numbers is worked out anew: kept over the loop, it
  // would cost the registers that the sums need
  auto renew = [](int& p, int& q) {
    asm volatile("" : "+v"(p), "+v"(q));
    if (MAKES_C) __builtin_amdgcn_sched_barrier(0);
  };
  // the own row of C (B) as an operand
  auto own_frag = [&](const T* base, int64_t ld, int kb) {
    const Frag<IO> f = frag8(base + (live ? own : 0) * ld + 32 * kb + 8 * g);
    return live ? f : frag_zero<IO>();
  };
  // B of tile i - d and C of tile i + d, where there are such, one after the other: f(d) multiplies them
  auto all_bc = [&](auto&& f) {
    typename LB::template Way<kMain> wb, wc;
    auto fetch = [&](int d, int t) {
      if (i - d >= 0) wb.load(Bg + (i - d) * kTile * a.b_row, a.b_row, 0, rows_in(i - d), t);
      if (i + d < ntiles) wc.load(Cg + (i + d) * kTile * a.c_row, a.c_row, 0, rows_in(i + d), t);
    };
    int t = tid;
    asm volatile("" : "+v"(t));
    fetch(0, t);
#pragma unroll
    for (int d = 0; d < kTiles; ++d) {
      __syncthreads();
      if (i - d >= 0) wb.store(lds + M::kB, t);
      if (i + d < ntiles) wc.store(lds + M::kC, t);
      __syncthreads();
      if (d < kLast) fetch(d + 1, t);
      f(d);
    }
    __syncthreads();
  };
  const char* const theirs = lds + (MAKES_C ? M::kB : M::kC);

  // a loader is half of the waves, or, with one buffer, all of them
  constexpr int kLoaders = M::kBufs == 2 ? kHalf : kMain;
  MainFill<IO, N, kLoaders> fill;
  const int lt = M::kBufs == 2 ? tid & (kHalf - 1) : tid;
  if (M::kBufs == 2 && LOADS) fill.load(a, pl, pl.h0, lt);

  // The own tile's tokens meet those of the tiles d = 0, 1, .. before it (dC) or behind it (dB, dx): of the first, the own
  // one, those up to the token (from it on). C . B of each, for all heads, and the sums over the heads. (Gh, Ph: of the
  // last tile behind it, for the other task.)
  float G[FAR + 1][4][4], P[FAR + 1][4][4], Gh[kHelps ? 4 : 1][4], Ph[kHelps ? 4 : 1][4];
  Frag<IO> bf[kNb];  // the own row of B
#pragma unroll
  for (int kb = 0; kb < kNb; ++kb) bf[kb] = own_frag(Bg, a.b_row, kb);
  {
    Frag<IO> cf[MAKES_C ? kNb : 1];
    if constexpr (MAKES_C)
#pragma unroll
      for (int kb = 0; kb < kNb; ++kb) cf[kb] = own_frag(Cg, a.c_row, kb);
    all_bc([&](int d) {
      int l = l15, gg = g;
      renew(l, gg);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (d <= FAR) {
#pragma unroll
          for (int kb = 0; kb < kNb; ++kb)
            v = mma(LB::row(theirs, 16 * q, 32 * kb, l, gg), MAKES_C ? cf[MAKES_C ? kb : 0] : bf[kb], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            G[d <= FAR ? d : 0][q][j] = v[j];
            P[d <= FAR ? d : 0][q][j] = 0.0f;
          }
        }
        if (kHelps && d == kLast) {
          v = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kb = 0; kb < kNb; ++kb) v = mma(LB::row(lds + M::kC, 16 * q, 32 * kb, l, gg), bf[kb], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            Gh[kHelps ? q : 0][j] = v[j];
            Ph[kHelps ? q : 0][j] = 0.0f;
          }
        }
      }
    });
  }
  if (M::kBufs == 2 && LOADS) fill.store(pl, lds, 0, lt);

  int buf = 0;
#pragma unroll 1
  for (int h = pl.h0; h < pl.h1; ++h) {
    const int64_t bch = bc * a.nheads + h;
    int t = lt, l = l15, gg = g;
    asm volatile("" : "+v"(t));
    renew(l, gg);
    __syncthreads();  // this head's tiles are whole, or (one buffer) the last one's have been read
    if constexpr (M::kBufs == 2) {
      if (LOADS) fill.load(a, pl, min(h + 1, pl.h1 - 1), t);
    } else {
      fill.load(a, pl, h, t);
      fill.store(pl, lds, 0, t);
      __syncthreads();
    }
    const MainTables& tab = reinterpret_cast<const MainTables*>(lds + M::kTab)[buf];
    const char* const toks = lds + buf * (M::kSlots * M::kX);
    const int me = i * kTile + 16 * w + l;  // the lane's token again
    const double cs_me = tab.cs[me];
    const char* const xi = toks + i * M::kX;
    const char* const yi = toks + (i + 1) * M::kX;
    f4* const dx_in = reinterpret_cast<f4*>(lds + M::kDx) + w * 256 + lane;  // of the lane's token, as accumulators lie
    float* const col_in = reinterpret_cast<float*>(lds + M::kCol) + w * 64 + lane;
    const float delta = own_delta(tab.delta[me]);
    Frag<IO> mine[2];  // the own row of dy (x)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) mine[kb] = LX::row(MAKES_C ? yi : xi, 16 * w, 32 * kb, l, gg);
    f4 dx[4];  // without delta and D: rows p = 16 pt + 4 g + j
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) dx[pt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    // dy . x of 32 others and the lane's token: rows of the others
    auto scores = [&](const char* other, int half, const Frag<IO>(&row)[2], f4(&m)[2]) {
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        m[o] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) m[o] = mma(LX::row(other, 32 * half + 16 * o, 32 * kb, l, gg), row[kb], m[o]);
      }
    };
    // what 32 others have of dx: their dy times C . B, weighted
    auto add_dx = [&](const char* other, int half, const f4(&gw)[2]) {
      const Wide<IO, 2> v = wide<IO, 2>(gw[0], gw[1]);
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) dx[pt] = mma_wide(LX::col_acc(other, 32 * half, 16 * pt, l, gg), v, dx[pt]);
    };
    // a half of tile i + d, d > 0, and the lane's token: its part of P, of the column of m (without delta) and of dx
    auto behind = [&](int d, int half, const Frag<IO>(&row)[2], float (*Gd)[4], float (*Pd)[4], float& column) {
      const int k = i + d;
      const char* const other = toks + (k + 1) * M::kX;
      const float er = decayed(tab.cs[k * kTile - 1] - cs_me);
      f4 m[2], gw[2];
      scores(other, half, row, m);
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int q = 2 * half + o, at = k * kTile + 16 * q + 4 * gg;
        const f4 wt = *reinterpret_cast<const f4*>(tab.from_end + at) * er;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool keep = !SEQ || at + j < next;
          const float cb = keep ? Gd[q][j] : 0.0f, mw = keep ? m[o][j] * wt[j] : 0.0f;
          gw[o][j] = !SEQ || keep ? cb * wt[j] : 0.0f;
          column = fmaf(mw, cb, column);
          Pd[q][j] = fmaf(mw, delta, Pd[q][j]);
        }
      }
      add_dx(other, half, gw);
      // summed here, not where the sums are used: the terms would wait in registers
#pragma unroll
      for (int q = 2 * half; q < 2 * half + 2; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(column), "+v"(Pd[q][j]));
    };
    // the own tile: a place of m has the same bits in its row and in its column, of which the step kernel takes one from
    // the other
    double in = 0.0;
    float all = 0.0f, skip = 0.0f;
    auto inside = [&](int half) {
      f4 m[2], gw[2];
      scores(MAKES_C ? xi : yi, half, mine, m);
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int q = 2 * half + o, at = i * kTile + 16 * q + 4 * gg;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = at + j;
          const float wt = decayed(MAKES_C ? cs_me - tab.cs[s] : tab.cs[s] - cs_me);
          const bool keep = MAKES_C ? s <= me && (!SEQ || s >= begin) : s >= me && (!SEQ || s < next);
          const float cb = keep ? G[0][q][j] : 0.0f, mw = m[o][j] * wt, with_delta = keep ? mw * (MAKES_C ? fabsf(tab.delta[s]) : delta) : 0.0f;
          in += s == me ? 0.0f : with_delta * cb;
          P[0][q][j] += with_delta;
          if (!MAKES_C) {
            skip = s == me ? m[o][j] : skip;
            all = fmaf(keep ? mw : 0.0f, cb, all);
            gw[o][j] = !SEQ || keep ? cb * wt : 0.0f;
          }
        }
      }
      if (!MAKES_C) add_dx(yi, half, gw);
#pragma unroll
      for (int q = 2 * half; q < 2 * half + 2; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(in), "+v"(all), "+v"(P[0][q][j]));
    };
    float* const tok = a.tok + bch * kQ + me;
    auto put_two = [&](float* to, int more, int less, double v) {
      const float m = static_cast<float>(v);
      to[more * a.tok_step] = m;
      to[less * a.tok_step] = static_cast<float>(v - m);
    };

    if constexpr (MAKES_C) {
      // what comes from the gradient behind the chunk, for the other task
      const bool open = !SEQ || next >= kQ;
      const float e = decayed(tab.cs[kQ - 1] - cs_me);
#pragma unroll
      for (int kb = 0; kb < kNb; ++kb) {
        if (IO == 0) renew(l, gg);
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) dx[pt] = mma_wide(LS::row(lds + M::kR, 16 * pt, 32 * kb, l, gg), bf[kb], dx[pt]);
      }
#pragma unroll
      for (int pt = 0; pt < 4; ++pt)
#pragma unroll
        for (int j = 0; j < 4; ++j) dx[pt][j] = open ? dx[pt][j] * e : 0.0f;
      if constexpr (kHelps) {
        Frag<IO> row[2];  // the own row of x
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) row[kb] = LX::row(xi, 16 * w, 32 * kb, l, gg);
        float column = 0.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          renew(l, gg);
          behind(kLast, half, row, Gh, Ph, column);
        }
        *col_in = column;
      }
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) dx_in[64 * pt] = dx[pt];
      __syncthreads();  // the other task's, and R has been read
      float out[FAR + 1] = {};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        renew(l, gg);
        inside(half);
      }
#pragma unroll
      for (int d = 1; d <= FAR; ++d) {
        const int k = i - d;
        const char* const other = toks + k * M::kX;
        const float er = decayed(cs_me - tab.cs[k * kTile + kTile - 1]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          renew(l, gg);
          f4 m[2];
          scores(other, half, mine, m);
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int q = 2 * half + o, at = k * kTile + 16 * q + 4 * gg;
            const f4 wt = *reinterpret_cast<const f4*>(tab.to_end + at) * er;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool keep = !SEQ || at + j >= begin;
              const float mw = keep ? m[o][j] * wt[j] : 0.0f;
              out[d] = fmaf(mw, keep ? G[d][q][j] : 0.0f, out[d]);
              P[d][q][j] += mw;
            }
          }
#pragma unroll
          for (int q = 2 * half; q < 2 * half + 2; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(out[d]), "+v"(P[d][q][j]));
        }
      }
      renew(l, gg);
      in = over_g(in);
      if (gg == 0) put_two(tok, kRowIn, kRowInLess, in);
#pragma unroll
      for (int d = 1; d <= FAR; ++d) {
        out[d] = over_g(out[d]);
        if (gg == 0) tok[(kRow1 + d - 1) * a.tok_step] = out[d];
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        renew(l, gg);
        inside(half);
      }
      float column = 0.0f;
      auto whole_behind = [&](int d) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          renew(l, gg);
          behind(d, half, mine, G[d], P[d], column);
        }
      };
      // a task that helps is there later
      constexpr int kBefore = HELP ? 1 : 0;
#pragma unroll
      for (int d = 1; d <= kBefore; ++d) whole_behind(d);
      __syncthreads();  // the other task has its part of dx
#pragma unroll
      for (int d = kBefore + 1; d <= FAR; ++d) whole_behind(d);
      renew(l, gg);
      if (HELP) column += *col_in;
      in = over_g(in);
      all = over_g(all);
      column = over_g(column);
      skip = over_g(skip);  // one lane has it
      const float D = tab.D;
      T* to = static_cast<T*>(a.dx) + ((row0 + me) * a.nheads + h) * kP + 4 * gg;
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) {
        const f4 yv = LX::four(yi, 16 * w + l, 16 * pt + 4 * gg), more = dx_in[64 * pt];
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(delta, dx[pt][j] + more[j], D * yv[j]);
        if (me < valid) {
          if constexpr (IO == 1) {
            *reinterpret_cast<u2*>(to + 16 * pt) = u2{round2(v[0], v[1]), round2(v[2], v[3])};
          } else {
            *reinterpret_cast<f4*>(to + 16 * pt) = v;
          }
        }
      }
      if (gg == 0) {
        put_two(tok, kColIn, kColInLess, in);
        tok[kColOut * a.tok_step] = delta * column;
        tok[kDirect * a.tok_step] = all + column;
        tok[kSkip * a.tok_step] = skip;
      }
    }
    if constexpr (M::kBufs == 2) {
      if (LOADS) fill.store(pl, lds, buf ^ 1, t);
      buf ^= 1;
    }
  }

  // the sums over the heads meet B and C, beside what the states carry
  const int64_t at = ((row0 + (live ? own : 0)) * a.ngroups + pl.grp) * N + 4 * g, whole = static_cast<int64_t>(a.batch) * a.seqlen * a.ngroups * N;
  f4 out[kNt];  // dC^T or dB^T: rows n = 16 nt + 4 g + j, the lane's token
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) out[nt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  if (pl.hs == 0)
    for (int k = 0; k < a.csplit; ++k) {
      const float* from = (MAKES_C ? a.dCc : a.dBc) + k * whole + at;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) out[nt] += *reinterpret_cast<const f4*>(from + 16 * nt);
    }
  f4 help[kHelps ? kNt : 1];
  auto times = [&](const char* tile, const float (*Pd)[4], f4* to) {
    int l = l15, gg = g;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      renew(l, gg);
      const float(&lo)[4] = Pd[2 * m], (&hi)[4] = Pd[2 * m + 1];
      const Wide<IO, 2> v = wide<IO, 2>(f4{lo[0], lo[1], lo[2], lo[3]}, f4{hi[0], hi[1], hi[2], hi[3]});
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) to[nt] = mma_wide(LB::col_acc(tile, 32 * m, 16 * nt, l, gg), v, to[nt]);
    }
  };
  all_bc([&](int d) {
    if (d <= FAR) times(theirs, P[d <= FAR ? d : 0], out);
    if constexpr (kHelps)
      if (d == kLast) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) help[nt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        times(lds + M::kC, Ph, help);
      }
  });
  if constexpr (HELP) {
    f4* const db = reinterpret_cast<f4*>(lds + M::kDB) + w * (64 * kNt) + lane;
    if constexpr (kHelps) {
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) db[64 * nt] = help[nt];
    }
    __syncthreads();
    if constexpr (!MAKES_C) {
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) out[nt] += db[64 * nt];
    }
  }
  if (!live) return;
  if (a.hsplit > 1) {
    float* to = (MAKES_C ? a.dCp : a.dBp) + pl.hs * whole + at;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) *reinterpret_cast<f4*>(to + 16 * nt) = out[nt];
    return;
  }
  T* to = static_cast<T*>(MAKES_C ? a.dC : a.dB) + at;
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) {
    if constexpr (IO == 1) {
      *reinterpret_cast<u2*>(to + 16 * nt) = u2{round2(out[nt][0], out[nt][1]), round2(out[nt][2], out[nt][3])};
    } else {
      *reinterpret_cast<f4*>(to + 16 * nt) = out[nt];
    }
  }
}

// 4. dB, dC, dx of 64 tokens, and what g and ddt are made of. Waves 0-3: dC of 16 tokens each; waves 4-7: dB and dx. Each
// task, for each number of tiles that it meets, is code of its own, so that its sums keep their registers.
template <int IO, int N, bool SEQ>
__global__ __launch_bounds__(kMain) void ssdb_main_kernel(const SbArgs a) {
  __shared__ __attribute__((aligned(512))) char lds[MainLds<IO, N>::kBytes];
  // the tiles of a chunk follow one another on one XCD: they read the same states and tokens
  MainPlace pl;
  {
    const int units = a.batch * a.nchunks * a.ngroups * a.hsplit;
    const int id = blockIdx.y * gridDim.x + blockIdx.x, j = id >> 3;
    pl.i = j % kTiles;
    int u = j / kTiles * 8 + (id & 7);
    if (u >= units) return;
    pl.hs = u % a.hsplit;
    u /= a.hsplit;
    pl.grp = u % a.ngroups;
    u /= a.ngroups;
    pl.c = u % a.nchunks;
    pl.b = u / a.nchunks;
  }
  pl.valid = min(kQ, a.seqlen - pl.c * kQ);
  if (pl.i * kTile >= pl.valid) return;  // the whole workgroup
  pl.ntiles = (pl.valid + kTile - 1) / kTile;
  const int rep = a.nheads / a.ngroups;
  pl.h0 = pl.grp * rep + pl.hs * a.per;
  pl.h1 = min(pl.h0 + a.per, (pl.grp + 1) * rep);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int far = pl.ntiles - 1 - pl.i;
  if (wave < 4) {
    if (IO == 1 && far == 3) return ssdb_task<IO, N, SEQ, true, 0, true, IO == 1>(a, pl, lds);
    switch (pl.i) {
      case 0: return ssdb_task<IO, N, SEQ, true, 0, true, false>(a, pl, lds);
      case 1: return ssdb_task<IO, N, SEQ, true, 1, true, false>(a, pl, lds);
      case 2: return ssdb_task<IO, N, SEQ, true, 2, true, false>(a, pl, lds);
      default: return ssdb_task<IO, N, SEQ, true, 3, false, false>(a, pl, lds);
    }
  }
  if (IO == 1 && pl.i == 3) return ssdb_task<IO, N, SEQ, false, 0, true, false>(a, pl, lds);
  switch (far) {
    case 0: return ssdb_task<IO, N, SEQ, false, 0, false, false>(a, pl, lds);
    case 1: return ssdb_task<IO, N, SEQ, false, 1, false, false>(a, pl, lds);
    case 2: return ssdb_task<IO, N, SEQ, false, 2, false, false>(a, pl, lds);
    default: return ssdb_task<IO, N, SEQ, false, IO == 1 ? 2 : 3, false, IO == 1>(a, pl, lds);
  }
}

// A running sum over a wave's lanes that starts again where a document begins.
__device__ __forceinline__ double run_lanes(double v, int cut, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double u = __shfl_up(v, o, 64);
    const int c = __shfl_up(cut, o, 64);
    if (lane >= o) {
      if (!cut) v += u;
      cut |= c;
    }
  }
  return v;
}

// Where a head's tokens hold what is not finite, the products of the main kernel may have met it times 0 at tokens that it is no
// term of. Their elements that are not finite are summed again here without the masked terms, by a wave for each token:
// dx of head h, and dB and dC of every rep-th token.
template <int IO, bool SEQ>
__device__ __forceinline__ void ssdb_mend(const SbArgs& a, int b, int c, int h) {
  using T = typename Io<IO>::T;
  const int lane = threadIdx.x & 63, n = a.d_state, rep = a.nheads / a.ngroups, grp = h / rep;
  const int valid = min(kQ, a.seqlen - c * kQ);
  const int64_t row0 = static_cast<int64_t>(b) * a.seqlen + static_cast<int64_t>(c) * kQ;
  const int64_t bc = static_cast<int64_t>(b) * a.nchunks + c;
  const T *const x = static_cast<const T*>(a.x) + row0 * a.x_row + lane, *const dy = static_cast<const T*>(a.dy) + row0 * a.dy_row + lane;
  const T *const B = static_cast<const T*>(a.B) + row0 * a.b_row + grp * n, *const C = static_cast<const T*>(a.C) + row0 * a.c_row + grp * n;
  auto wrong = [](float v) { return !(fabsf(v) < INFINITY); };
  for (int t = threadIdx.x >> 6; t < valid; t += kQ / 64) {
    const int first = SEQ ? max(a.begin[bc * kQ + t], 0) : 0, next = SEQ ? a.next[bc * kQ + t] : kQ, last = min(next, valid);
    {
      const int64_t bch = bc * a.nheads + h;
      const double* cs = a.cs + bch * kQ;
      T* const to = static_cast<T*>(a.dx) + ((row0 + t) * a.nheads + h) * kP + lane;
      const bool mine = wrong(Io<IO>::load(to));
      if (__any(mine)) {
        float sum = 0.0f;
        for (int r = t; r < last; ++r) {
          float cb = 0.0f;
          for (int k = lane; k < n; k += 64) cb = fmaf(Io<IO>::load(C + r * a.c_row + k), Io<IO>::load(B + t * a.b_row + k), cb);
          sum = fmaf(decayed(cs[r] - cs[t]) * lanes_sum(cb, 64), Io<IO>::load(dy + r * a.dy_row + h * kP), sum);
        }
        if (next >= kQ) {
          const float* R = a.R + (bch * kP + lane) * n;
          float rb = 0.0f;
          for (int k = 0; k < n; ++k) rb = fmaf(R[k], Io<IO>::load(B + t * a.b_row + k), rb);
          sum = fmaf(decayed(cs[kQ - 1] - cs[t]), rb, sum);
        }
        if (mine) Io<IO>::store(to, fmaf(own_delta(a.delta[bch * kQ + t]), sum, a.D[h] * Io<IO>::load(dy + t * a.dy_row + h * kP)));
      }
    }
    if (t % rep != h % rep) continue;
    const int64_t row = ((row0 + t) * a.ngroups + grp) * n, whole = static_cast<int64_t>(a.batch) * a.seqlen * a.ngroups * n;
    for (int of_c = 0; of_c < 2; ++of_c) {
      T* const to = static_cast<T*>(of_c ? a.dC : a.dB) + row;
      const float* const from = (of_c ? a.dCc : a.dBc) + row;
      bool mine[2];
      float sum[2] = {0.0f, 0.0f};
      for (int i = 0; i < 2; ++i) {
        const int k = lane + 64 * i;
        mine[i] = k < n && wrong(Io<IO>::load(to + k));
        if (mine[i])
          for (int j = 0; j < a.csplit; ++j) sum[i] += from[j * whole + k];
      }
      if (!__any(mine[0] || mine[1])) continue;
      for (int hh = grp * rep; hh < (grp + 1) * rep; ++hh) {
        const int64_t bch = bc * a.nheads + hh;
        const double* cs = a.cs + bch * kQ;
        const float own = Io<IO>::load((of_c ? dy + t * a.dy_row : x + t * a.x_row) + hh * kP);
        for (int o = of_c ? first : t; o < (of_c ? t + 1 : last); ++o) {
          const float m = lanes_sum(own * Io<IO>::load((of_c ? x + o * a.x_row : dy + o * a.dy_row) + hh * kP), 64);
          const float w = decayed(of_c ? cs[t] - cs[o] : cs[o] - cs[t]) * (of_c ? fabsf(a.delta[bch * kQ + o]) : own_delta(a.delta[bch * kQ + t])) * m;
          for (int i = 0; i < 2; ++i) {
            const int k = lane + 64 * i;
            if (k < n) sum[i] = fmaf(w, Io<IO>::load((of_c ? B + o * a.b_row : C + o * a.c_row) + k), sum[i]);
          }
        }
      }
      for (int i = 0; i < 2; ++i)
        if (mine[i]) Io<IO>::store(to + lane + 64 * i, sum[i]);
    }
  }
}

// 5. g and ddt of a chunk's tokens, and the chunk's sums for dA, ddt_bias and dD. A wave has a tile.
template <int IO, bool SEQ>
__global__ __launch_bounds__(kQ) void ssdb_step_kernel(const SbArgs a) {
  using T = typename Io<IO>::T;
  __shared__ double of_s[kTiles], of_r[kTiles], pair[kTiles][kTiles];  // sums of tiles, and of m over two tiles
  __shared__ double sums[3][kTiles];
  const int tid = threadIdx.x, lane = tid & 63, tile = tid >> 6, c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int valid = min(kQ, a.seqlen - c * kQ);
  const int64_t bc = static_cast<int64_t>(b) * a.nchunks + c, bch = bc * a.nheads + h;
  const int64_t row = static_cast<int64_t>(b) * a.seqlen + static_cast<int64_t>(c) * kQ + tid;
  const int m = tile * kTile + kTile - 1 - lane;  // from the tile's last token on
  auto tok = [&](int n, int t) { return t < valid ? a.tok[n * a.tok_step + bch * kQ + t] : 0.0f; };
  auto two = [&](int more, int less) { return static_cast<double>(tok(more, m)) + tok(less, m); };
  const float any_delta = a.delta[bch * kQ + tid], delta = own_delta(any_delta);
  const bool gone = static_cast<double>(fabsf(any_delta)) * a.A[h] <= kGone;  // at this token, whose g is 0 times what it would be
  const bool gone_m = __shfl(static_cast<int>(gone), 63 - lane), gone_next = __shfl(static_cast<int>(gone), (64 - lane) & 63);
  // inside the tile; no term reaches over a document's begin, or over a step of which nothing is left
  const bool cut_m = lane > 0 && (gone_next || (SEQ && a.next[bc * kQ + m] == m + 1));
  const double row_m = two(kRowIn, kRowInLess);
  double down = run_lanes(row_m - two(kColIn, kColInLess), cut_m, lane);
  // from tiles before it, and from S
  double late = 0.0;
  for (int d = 1; d <= tile; ++d) {
    const float v = tok(kRow1 + d - 1, m);
    late += v;
    double s = v;
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) pair[tile][tile - d] = s;
  }
  const float raw_s = tok(kOfS, m), raw_r = tok(kOfR, tid);
  const double s_m = !SEQ || a.begin[bc * kQ + m] < 0 ? raw_s : 0.0f;
  down += run_lanes(late, 0, lane);
  const double from_s = run_lanes(s_m, 0, lane);
  if (lane == 63) of_s[tile] = from_s;
  // (the token's own row is 0 times what is before it)
  down = __shfl(gone_m ? row_m + late + s_m : down + from_s, 63 - lane, 64);  // turned round
  // with tiles behind it, and from R: of the tokens before this one
  // (0 where nothing behind the tile, or behind the chunk, is of the token's document, whatever its delta)
  const int next = SEQ ? a.next[bc * kQ + tid] : kQ;
  const float of_r0 = !SEQ || next >= kQ ? raw_r : 0.0f;
  const double col = !SEQ || next > (tid | (kTile - 1)) ? tok(kColOut, tid) : 0.0f;
  const double r = !SEQ || next >= kQ ? static_cast<double>(of_r0) * delta : 0.0;
  const double upto = run_lanes(col + r, 0, lane), before = __shfl_up(upto, 1, 64);
  const double from_r = run_lanes(r, 0, lane);
  if (lane == 63) of_r[tile] = from_r;
  __syncthreads();
  double g = lane > 0 ? down + before : down;
  for (int j = 0; j < kTiles; ++j) {
    if (j > tile) g += of_s[j];
    if (j < tile) g += of_r[j];
    if (j > tile)
      for (int k = 0; k < tile; ++k) g += pair[j][k];
  }
  const float decay = a.decay[bch];
  if (!(decay < 0.0f)) {
    double whole = 0.0;
    for (int i = 0; i < 16; ++i) whole += a.dot[bch * 16 + i];
    g += whole * decay;
  }
  if (gone) g = down;
  if (SEQ && a.begin[bc * kQ + tid] == tid) g = 0.0;  // nothing reaches a document's first token
  double all[3] = {};  // of dA, ddt_bias and dD: terms of either sign, many of which cancel
  if (tid < valid) {
    const float v = Io<IO>::load(static_cast<const T*>(a.dt) + row * a.dt_row + h) + a.dt_bias[h];
    double d = (static_cast<double>(a.A[h]) * g + (static_cast<double>(tok(kDirect, tid)) + of_r0)) * (1.0f / (1.0f + expf(-v)));
    if (delta != delta) d = delta;  // all that this token is a term of meets a step that is NaN
    Io<IO>::store(static_cast<T*>(a.ddt) + row * a.nheads + h, static_cast<float>(d));
    all[0] = g * delta;
    all[1] = d;
    all[2] = tok(kSkip, tid);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    for (int o = 32; o > 0; o >>= 1) all[i] += __shfl_xor(all[i], o, 64);
    if (lane == 0) sums[i][tile] = all[i];
  }
  __syncthreads();
  if (tid < 3) {  // rounded once a chunk, as the outputs are; the chunks' sums are added in float32
    float* to = tid == 0 ? a.pA : tid == 1 ? a.pb : a.pD;
    to[bch] = static_cast<float>((sums[tid][0] + sums[tid][1]) + (sums[tid][2] + sums[tid][3]));
  }
  // a token's shares are not finite where its x, dy, B or C are not: infinity, or 0 times it, is in them
  if (__syncthreads_or(!(fabsf(raw_s) < INFINITY && fabsf(raw_r) < INFINITY))) ssdb_mend<IO, SEQ>(a, b, c, h);
}

// dB and dC of the splits of the heads, one after the other.
template <int IO>
__global__ __launch_bounds__(256) void ssdb_join_kernel(int64_t n4, int32_t splits, const float* __restrict__ dBp,
                                                       const float* __restrict__ dCp, typename Io<IO>::T* dB,
                                                       typename Io<IO>::T* dC) {
  const float* from = blockIdx.y == 0 ? dBp : dCp;
  auto* to = blockIdx.y == 0 ? dB : dC;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n4; i += static_cast<int64_t>(gridDim.x) * 256) {
    f4 s = reinterpret_cast<const f4*>(from)[i];
    for (int k = 1; k < splits; ++k) s += reinterpret_cast<const f4*>(from)[k * n4 + i];
#pragma unroll
    for (int j = 0; j < 4; ++j) Io<IO>::store(to + 4 * i + j, s[j]);
  }
}

// Workgroups that share the heads of a group: as many as end first. One takes a CU for itself, and a time of `fixed` heads
// before and behind its own. (A chunk has kTiles of the main kernel, and two of the carry kernel; in float32 it has four,
// which are planned as two. Twelve heads in three
// groups, 2 x 1501 tokens, float32: split in two, which is 288 workgroups, the main kernel took 124 us and a kernel to join them 5, whole 95.)
int heads_split(int32_t batch, int32_t nchunks, int32_t nheads, int32_t ngroups, int of_chunk, int fixed) {
  const int rep = nheads / ngroups;
  const int64_t units = static_cast<int64_t>(batch) * nchunks * ngroups * of_chunk;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= rep && (n == 1 || units * n <= 1024); ++n) {
    const int per = (rep + n - 1) / n;
    if ((rep + per - 1) / per != n) continue;
    const int64_t time = (units * n + 255) / 256 * (fixed + per);
    if (time < least) {
      least = time;
      best = n;
    }
  }
  return best;
}

struct Ws {
  size_t S, R, decay, cs, delta, begin, next, dot, tok, dBp, dCp, dBc, dCc, pA, pb, pD, total, tok_step;
};
Ws layout(int32_t batch, int32_t seqlen, int32_t nheads, int32_t d_state, int32_t ngroups) {
  Ws w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t nchunks = (static_cast<size_t>(seqlen) + kQ - 1) / kQ, bc = batch * nchunks, bch = bc * nheads;
  const size_t split = heads_split(batch, static_cast<int32_t>(nchunks), nheads, ngroups, kTiles, 4);
  const size_t csplit = heads_split(batch, static_cast<int32_t>(nchunks), nheads, ngroups, 2, 2);
  const size_t one = static_cast<size_t>(batch) * seqlen * ngroups * static_cast<size_t>(d_state) * 4, part = split > 1 ? split * one : 0;
  w.S = take(bch * kP * d_state * 4);
  w.R = take(bch * kP * d_state * 4);
  w.decay = take(bch * 4);
  w.cs = take(bch * kQ * 8);
  w.delta = take(bch * kQ * 4);
  w.begin = take(bc * kQ * 4);
  w.next = take(bc * kQ * 4);
  w.dot = take(bch * 16 * 4);
  w.tok = take(bch * kQ * 4 * kTokSums);
  w.tok_step = bch * kQ;
  w.dBp = take(part);
  w.dCp = take(part);
  w.dBc = take(csplit * one);
  w.dCc = take(csplit * one);
  w.pA = take(bch * 4);
  w.pb = take(bch * 4);
  w.pD = take(bch * 4);
  w.total = at;
  return w;
}

// n workgroups, and some more that find nothing to do: at most 2^22 along x (a dispatch dimension counts its work-items in
// 32 bits), the rest along y.
dim3 grid_of(int64_t n) {
  const int64_t gx = std::min(n, int64_t{1} << 22);
  return dim3(static_cast<unsigned>(gx), static_cast<unsigned>((n + gx - 1) / gx));
}

template <int IO, int N, bool SEQ>
hipError_t launch_typed(const SsdBwdCall& c, const SbArgs& a) {
  hipError_t e;
  hipLaunchKernelGGL((ssdb_state_kernel<IO, N, SEQ>), dim3(2 * a.nchunks, a.nheads, a.batch), dim3(kState), 0, c.stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int n4 = kP * N / 4;
  hipLaunchKernelGGL(ssdb_pass_kernel, dim3(2 * (n4 / kState), a.nheads, a.batch), dim3(kState), 0, c.stream, a, n4);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t groups = static_cast<int64_t>(a.batch) * a.nchunks * a.ngroups, units = groups * a.hsplit;
  hipLaunchKernelGGL((ssdb_carry_kernel<IO, N, SEQ>), grid_of(groups * a.csplit * 2 * (kQ / CarryLds<IO, N>::kRows)), dim3(kMain), 0,
                     c.stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((ssdb_main_kernel<IO, N, SEQ>), grid_of((units + 7) / 8 * 8 * kTiles), dim3(kMain), 0, c.stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.hsplit > 1) {
    using T = typename Io<IO>::T;
    const int64_t n4 = static_cast<int64_t>(a.batch) * a.seqlen * a.ngroups * N / 4;
    hipLaunchKernelGGL(ssdb_join_kernel<IO>, dim3(static_cast<unsigned>(std::min<int64_t>((n4 + 255) / 256, 65536)), 2), dim3(256),
                       0, c.stream, n4, a.hsplit, a.dBp, a.dCp, static_cast<T*>(a.dB), static_cast<T*>(a.dC));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssdb_step_kernel<IO, SEQ>), dim3(a.nchunks, a.nheads, a.batch), dim3(kQ), 0, c.stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int nblk = a.batch * a.nchunks;
  return launch_part_sums(nblk, {{a.nheads, a.pA, a.dA}, {a.nheads, a.pb, a.ddt_bias}, {a.nheads, a.pD, a.dD}}, c.stream);
}

template <int IO, int N>
hipError_t launch_seq(const SsdBwdCall& c, const SbArgs& a) {
  return c.seq_idx ? launch_typed<IO, N, true>(c, a) : launch_typed<IO, N, false>(c, a);
}

}  // namespace

size_t ssd_bwd_ws_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t d_state, int32_t ngroups) {
  return layout(batch, seqlen, nheads, d_state, ngroups).total;
}

hipError_t launch_ssd_bwd(const SsdBwdCall& c) {
  const Ws w = layout(c.batch, c.seqlen, c.nheads, c.d_state, c.ngroups);
  SbArgs a{};
  a.batch = c.batch;
  a.seqlen = c.seqlen;
  a.nheads = c.nheads;
  a.ngroups = c.ngroups;
  a.d_state = c.d_state;
  a.nchunks = (c.seqlen + kQ - 1) / kQ;
  a.hsplit = heads_split(c.batch, a.nchunks, c.nheads, c.ngroups, kTiles, 4);
  a.per = (c.nheads / c.ngroups + a.hsplit - 1) / a.hsplit;
  a.csplit = heads_split(c.batch, a.nchunks, c.nheads, c.ngroups, 2, 2);
  a.cper = (c.nheads / c.ngroups + a.csplit - 1) / a.csplit;
  a.x_row = c.x_row;
  a.dt_row = c.dt_row;
  a.b_row = c.b_row;
  a.c_row = c.c_row;
  a.dy_row = c.dy_row;
  a.x = c.x;
  a.dt = c.dt;
  a.B = c.B;
  a.C = c.C;
  a.dy = c.dy;
  a.seq_idx = c.seq_idx;
  a.dt_bias = c.dt_bias;
  a.A = c.A;
  a.D = c.D;
  a.state_in = c.state_in;
  a.dstate_out = c.dstate_out;
  a.dx = c.dx;
  a.ddt = c.ddt;
  a.dB = c.dB;
  a.dC = c.dC;
  a.ddt_bias = c.ddt_bias;
  a.dA = c.dA;
  a.dD = c.dD;
  a.dstate_in = c.dstate_in;
  auto f = [&](size_t at) { return reinterpret_cast<float*>(c.workspace + at); };
  a.S = f(w.S);
  a.R = f(w.R);
  a.decay = f(w.decay);
  a.cs = reinterpret_cast<double*>(c.workspace + w.cs);
  a.delta = f(w.delta);
  a.begin = reinterpret_cast<int32_t*>(c.workspace + w.begin);
  a.next = reinterpret_cast<int32_t*>(c.workspace + w.next);
  a.dot = f(w.dot);
  a.tok = f(w.tok);
  a.tok_step = static_cast<int64_t>(w.tok_step);
  a.dBp = f(w.dBp);
  a.dCp = f(w.dCp);
  a.dBc = f(w.dBc);
  a.dCc = f(w.dCc);
  a.pA = f(w.pA);
  a.pb = f(w.pb);
  a.pD = f(w.pD);
  if (c.io_dtype == 0) return c.d_state == 64 ? launch_seq<0, 64>(c, a) : launch_seq<0, 128>(c, a);
  return c.d_state == 64 ? launch_seq<1, 64>(c, a) : launch_seq<1, 128>(c, a);
}

}  // namespace mscan
