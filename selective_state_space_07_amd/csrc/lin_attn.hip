// Linear attention with a fixed decay for each head, on the matrix cores.
//
// Per batch row and head, with lam = exp(log_decay[h]) and a state S[d_v][d_k]:
//   S_t = lam S_{t-1} + v_t k_t^T,   y_t = scale S_t q_t.
// Over a chunk of 64 tokens, numbered from 0, with the state S before it, this
// is (up to rounding)
//   y_t  = scale [ sum_{s<=t} lam^(t-s) (q_t . k_s) v_s + lam^(t+1) S q_t ],
//   S'   = lam^64 S + sum_s lam^(63-s) v_s k_s^T.
// The gradients are the same sums with the operands exchanged. With
// R_t = lam R_{t+1} + scale dy_t q_t^T (from the last token to the first),
//   dq_t = scale S_t^T dy_t: the sum over (q, k, v) := (dy, v, k),
//   dk_t = R_t^T v_t:        the reversed sum over (v, dy, q),
//   dv_t = R_t k_t:          the reversed sum over (k, q, dy),
// so one kernel serves both directions; a backward call is its three roles in
// one launch. The incoming state of a reversed sum (the gradient of the final
// state) stands at its first token, not one step before it: `off` is 0 there,
// in lam^(t+off) and lam^(64-off-s).
//
// A workgroup walks the chunks of one (batch row, head, 64 columns of v) in
// order, eight waves with two tasks. Four of them own 16 tokens of the chunk
// each and make y: A^T = K Q^T (the scores, which stay in registers: the rows
// of its 16x16 tiles are numbered, by `spread`, so that the accumulators of
// two tiles are the next product's operand as they stand), then
// y^T = S Q^T + V^T A^T. The other four own 16 columns of v each and keep the
// state of theirs in accumulators, S^T += K^T (w V), from the first chunk to
// the last; each chunk's starting state goes to the first four through LDS.
// Both tasks of a chunk run at once, one wave of each on a SIMD, and with K, V
// and S in LDS twice there is one barrier to a chunk. K and V come through
// registers two chunks ahead (one where the registers do not suffice), Q
// straight into the lanes that multiply it. A chunk is bound by the issue of
// its instructions, so places in memory are worked out once for all chunks.
//
// float32 io runs on the bfloat16 matrix cores as well, sixteen times as fast
// as the float32 ones: every operand is the sum of three bfloat16 parts of 8
// significant bits each, which hold a float32 whole, and a product takes its
// six largest products of parts (the next are below 2^-23 of it).
//
// For bfloat16 io the scores and the state, float32 values that meet operands of
// 8 significant bits, are two parts each: 16 bits, so that y has the error of its
// own rounding alone, 1.66e-3 of itself in the mean. With one part each that was
// 2.35e-3, at 58 us instead of 73 for 8 x 2048 tokens, 12 heads of 128, and 155
// instead of 193 for the gradients.
//
// Measured on an MI355X, where a large copy reaches 5.2 TB/s: 8 x 2048 tokens,
// 12 heads of 128, bfloat16: 73 us (201 MB to read and write, 2.8 TB/s), the
// gradients 193 us (352 MB, 1.8 TB/s: 576 workgroups are two and a quarter
// rounds of 256 CUs and take three). Both are bound by the issue of instructions
// (of the 4900 cycles of a chunk the gradients' vector instructions take 1870 on
// each SIMD and the matrix ones 1490): without the state's products they take 64
// and 175 us, without y's 63 and 173, without either 58 and 162, without the
// traffic of K, V, Q and y 64 and 181. With one part of scores and state each,
// one task after the other, four barriers a chunk and bank conflicts took 209 us
// instead of 58, and four chunks ahead instead of two changed nothing (58 and
// 161 us). Two workgroups on a CU would need 80 KB of LDS each, not 116, and 128
// registers a lane, not 170.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linattn_internal.h"
#include "mfma_frag.h"
#include "scan_device.h"

namespace mscan {

namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kVS = 64;        // columns of v per workgroup
constexpr int kThreads = 256;  // four waves of 16 columns: the state's task
constexpr int kMaxRoles = 3;

struct LaArgs {
  int32_t batch, seqlen, nheads, ngroups, nseg, seg_chunks, nroles, nsl;  // nsl: column slices of the widest role
  int32_t nslices;                                                         // of all roles
  const int32_t* seq_idx;
  const float* log_decay;
  float* ws;         // segment states
  int32_t* flags;    // [role][batch][nseg]: a document begins inside the segment or at its start
  LaRole role[kMaxRoles];
};

// lam^n for whole n >= 0 (1 for n = 0 also where lam is 0); g2 = log2(lam)
__device__ __forceinline__ float power(float g2, int n) {
  return n == 0 ? 1.0f : exp2_hw(static_cast<float>(n) * g2);
}

// 8 k-values of a matrix-core operand, each the sum of N bfloat16 parts.
template <int N>
struct Parts {
  bf8 p[N];
};
// An operand of the io type: bfloat16 is one part, float32 three.
template <int IO>
using Op = Parts<IO == 1 ? 1 : 3>;
// A float32 value that is multiplied with one: a score, or the state.
template <int IO>
using Sum = Parts<IO == 1 ? 2 : 3>;

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
// Two values as one word of bfloat16, rounded, or (as the first of several parts)
// cut: rounding would take finite values beyond 3.38e38 to infinity.
__device__ __forceinline__ uint32_t round2(float a, float b) {
  uint32_t w = __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
  asm("" : "+v"(w));  // or the compiler would round the two one by one, to unpack them from there
  return w;
}
__device__ __forceinline__ uint32_t cut2(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// What a part left of two values, exactly: the next part is made of that.
__device__ __forceinline__ void rest2(float& a, float& b, uint32_t w) {
  a -= __uint_as_float(w << 16);
  b -= __uint_as_float(w & 0xFFFF0000u);
}
template <bool CUT>
__device__ __forceinline__ u4 pack(const float (&x)[8]) {
  u4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = CUT ? cut2(x[2 * j], x[2 * j + 1]) : round2(x[2 * j], x[2 * j + 1]);
  return w;
}
__device__ __forceinline__ void rest(float (&x)[8], u4 w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t e = w[j];
    rest2(x[2 * j], x[2 * j + 1], e);
  }
}
// NaN once any value in w is infinite or NaN
__device__ __forceinline__ float unfit(u4 w, float so_far) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t e = w[j];
    so_far = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2, e), bf2{}, so_far, false);
  }
  return so_far;
}
template <int N>
__device__ __forceinline__ Parts<N> split(f4 lo, f4 hi) {
  float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Parts<N> o;
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const u4 w = p == 0 && N > 1 ? pack<true>(x) : pack<false>(x);
    o.p[p] = __builtin_bit_cast(bf8, w);
    rest(x, w);
  }
  return o;
}
// The same of four values, two to a word; where none is beyond 3.38e38 the first
// part may be rounded, which leaves the last of two a quarter of the error.
template <bool CUT, int N>
__device__ __forceinline__ void split4(f4 v, u2 (&o)[N]) {
  float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < N; ++p) {
    const bool cut = CUT && p == 0 && N > 1;
    const uint32_t a = cut ? cut2(x[0], x[1]) : round2(x[0], x[1]), b = cut ? cut2(x[2], x[3]) : round2(x[2], x[3]);
    o[p] = u2{a, b};
    rest2(x[0], x[1], a);
    rest2(x[2], x[3], b);
  }
}
// Element j as float32.
template <int N>
__device__ __forceinline__ float get(const Parts<N>& f, int j) {
  float v = static_cast<float>(f.p[N - 1][j]);
#pragma unroll
  for (int p = N - 2; p >= 0; --p) v += static_cast<float>(f.p[p][j]);
  return v;
}
// A lane's eight k-values where `mask` has their bits, 0 elsewhere.
template <int N>
__device__ __forceinline__ Parts<N> masked(const Parts<N>& f, u4 mask) {
  Parts<N> o;
#pragma unroll
  for (int p = 0; p < N; ++p) o.p[p] = __builtin_bit_cast(bf8, __builtin_bit_cast(u4, f.p[p]) & mask);
  return o;
}
// Those from `first` to `last`.
template <int N>
__device__ __forceinline__ Parts<N> between(const Parts<N>& f, int first, int last) {
  u4 mask;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mask[j] = ((2 * j >= first) & (2 * j <= last) ? 0xFFFFu : 0u) |
              ((2 * j + 1 >= first) & (2 * j + 1 <= last) ? 0xFFFF0000u : 0u);
  return masked(f, mask);
}
// Where they are finite: elsewhere the first part is not.
template <int N>
__device__ __forceinline__ u4 finite(const Parts<N>& f) {
  const u4 w = __builtin_bit_cast(u4, f.p[0]);
  u4 mask;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mask[j] = ((w[j] & 0x7F80u) != 0x7F80u ? 0xFFFFu : 0u) | ((w[j] & 0x7F800000u) != 0x7F800000u ? 0xFFFF0000u : 0u);
  return mask;
}
// An infinity or NaN whole in its first part: the rests of it are NaN, and 0 here.
template <int N>
__device__ __forceinline__ Parts<N> whole(const Parts<N>& f) {
  Parts<N> o = masked(f, finite(f));
  o.p[0] = f.p[0];
  return o;
}
// acc[i] += a[i] b over the pairs of parts that matter, the smallest first, and
// each pair for all i in turn: consecutive products do not wait for each other.
template <int M, int NA, int NB>
__device__ __forceinline__ void mma_each(f4* acc, const Parts<NA> (&a)[M], const Parts<NB>& b) {
  constexpr int kMost = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int o = kMost; o >= 0; --o)
#pragma unroll
    for (int pa = 0; pa < NA; ++pa) {
      const int pb = o - pa;
      if (pb < 0 || pb >= NB) continue;
#pragma unroll
      for (int i = 0; i < M; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i].p[pa], b.p[pb], acc[i], 0, 0, 0);
    }
}

// The operand that two neighbouring tiles of accumulators are: 8 consecutive
// rows, of which the first tile has the upper four where g is odd.
template <int N>
__device__ __forceinline__ Parts<N> tiles_op(f4 even, f4 odd, int g) {
  const bool up = g & 1;
  if constexpr (N == 1) {
    const u4 v = __builtin_bit_cast(u4, frag_regs<1>(even, odd).v);
    const u4 w = {up ? v.z : v.x, up ? v.w : v.y, up ? v.x : v.z, up ? v.y : v.w};
    return Parts<1>{{__builtin_bit_cast(bf8, w)}};
  } else {
    return split<N>(up ? odd : even, up ? even : odd);
  }
}

// The column (of a tile, or of the state) that row or column m of a wave's i-th
// 16-wide product stands for. Two neighbouring i share 32 columns: m / 4 = c
// has columns 8 c .. 8 c + 3 of them in one and 8 c + 4 .. 8 c + 7 in the other,
// the lower four first for even c (so that one transposed read takes both
// halves of the 16-byte pieces, and with them all banks).
__device__ __forceinline__ int spread(int i, int m) {
  const int c = m >> 2;
  return 32 * (i >> 1) + 8 * c + 4 * ((i ^ c) & 1) + (m & 3);
}

// `off` where ok, else an offset beyond any buffer range. Without a branch:
// the compiler would put the load or store behind it.
__device__ __forceinline__ uint32_t in_range(uint32_t off, bool ok) {
  return off | ((static_cast<uint32_t>(ok) - 1u) & 0xFFFFFFC0u);
}
// The rows of a chunk lie upwards in memory, or downwards where the sum runs
// from the last token to the first. `low` is the row that lies lowest; row r of
// a whole chunk is at far(r) * stride from it, and in a last chunk of n rows
// that runs downwards all of them are cut(n) * stride nearer. Rows from n on
// are then out of the range of the buffer, above it or (as unsigned numbers)
// below 0: strides are at most 2^26 bytes.
struct Order {
  bool rev;
  __device__ __forceinline__ uint32_t far(int r) const { return static_cast<uint32_t>(rev ? kC - 1 - r : r); }
  __device__ __forceinline__ uint32_t cut(int n) const { return static_cast<uint32_t>(rev ? kC - n : 0); }
  __device__ __forceinline__ int64_t low(int n) const { return rev ? n - 1 : 0; }  // in rows from the first
};
// A matrix of which a workgroup walks the chunks: the first token's row, the
// bytes from a row to the next one in memory, and those of a row that are read.
struct Rows {
  const char* p;
  uint32_t stride, width;
  Order order;
  // n rows from chunk c on; none are in range where n <= 0. No branch may stand
  // around a load: behind one the compiler could not tell the loads in flight
  // apart and would wait for all of them.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int c, int n) const {
    const int64_t row = static_cast<int64_t>(c) * kC + order.low(n);
    const char* at = p + (order.rev ? -row : row) * stride;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0,
                                             n > 0 ? stride * static_cast<uint32_t>(n - 1) + width : 0, 0x00020000);
  }
};

// A 64-row tile of W columns in LDS and its way there from global memory
// through registers (the load is issued a chunk ahead).
//
// The 16-byte pieces of a row are exchanged by an exclusive-or with a number
// made of the row's low bits, so that each way of reading hits every bank
// once: one piece of the 16 rows spread(i, .), and, in half a wave of
// transposed reads, rows 0-3 and 8-11 of four half pieces.
//
// All reads are (base ^ constant) + constant with a base that depends on the
// lane alone: a step along the row changes bits that the exchange leaves to
// the exclusive-or, and 4 or 32 rows further the exchange is the same.
// A tile of several parts lies there as that many bfloat16 tiles.
template <int IO, int W, int NT, typename OP = Op<IO>>
struct Tile {
  using T = typename Io<IO>::T;
  static constexpr int kParts = sizeof(OP) / sizeof(bf8);
  static constexpr uint32_t kRow = W * 2, kPart = kC * kRow, kBytes = kParts * kPart;  // bytes in LDS
  static constexpr int kPer = W * sizeof(T) / 16;  // 16-byte pieces of a row in memory
  static constexpr int kN = kC * kPer / NT;        // pieces of a thread
  u4 v[kN];

  static __device__ __forceinline__ uint32_t exchange(int row) {
    // 8 pieces a row: two rows span the banks, so the row's lowest bit is left
    // out; bit 2 is, for its rows are read apart; bits 1 and 3 must not meet
    // in bit 1, which tells the half pieces of one transposed read apart
    const int x = ((row >> 1) & 1) | ((row >> 3) & 2) | ((row >> 1) & 4);  // row bits 1, 4, 3
    return W == 64 ? x : ((x & 1) << 2) | (x & 2) | ((x & 4) << 1) | (row & 1);
  }
  // Where element `col` of a row lies in each part.
  static __device__ __forceinline__ uint32_t at(int row, int col) {
    return static_cast<uint32_t>(row) * kRow + (static_cast<uint32_t>(2 * col) ^ (exchange(row) << 4));
  }
  // The places of a thread's pieces in a whole chunk; those of columns that
  // are not read are out of every range.
  struct Ways {
    uint32_t at[kN];
    __device__ __forceinline__ Ways(const Rows& m, uint32_t tid) {
      const uint32_t c = tid % kPer * 16;  // one column, NT / kPer rows apart
#pragma unroll
      for (int q = 0; q < kN; ++q)
        at[q] = in_range(m.order.far(static_cast<int>(tid / kPer) + q * (NT / kPer)) * m.stride + c, c < m.width);
    }
  };
  // n rows of a chunk; 0 behind them and beyond the columns
  __device__ __forceinline__ void load(const Rows& m, const Ways& w, int c, int n) {
    const auto rsrc = m.chunk(c, n);
    const uint32_t cut = m.order.cut(n) * m.stride;
#pragma unroll
    for (int q = 0; q < kN; ++q)
      v[q] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, w.at[q] - cut, 0, 0));
  }
  __device__ __forceinline__ void store(char* lds, uint32_t tid) const {
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      char* p = lds + at(tid / kPer + q * (NT / kPer), tid % kPer * (16 / sizeof(T)));
      if constexpr (IO == 1) {
        *reinterpret_cast<u4*>(p) = v[q];
      } else {
        put4<true>(p, __builtin_bit_cast(f4, v[q]));
      }
    }
  }
  // Four neighbouring elements, split into the parts.
  template <bool CUT>
  static __device__ __forceinline__ void put4(char* p, f4 x) {
    u2 o[kParts];
    split4<CUT>(x, o);
#pragma unroll
    for (int i = 0; i < kParts; ++i) *reinterpret_cast<u2*>(p + i * kPart) = o[i];
  }
  static __device__ __forceinline__ f4 get4(const char* lds, int row, int col) {
    f4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = kParts - 1; i >= 0; --i) {
      const u2 o = *reinterpret_cast<const u2*>(lds + at(row, col) + i * kPart);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        x[2 * r] += __uint_as_float(o[r] << 16);
        x[2 * r + 1] += __uint_as_float(o[r] & 0xFFFF0000u);
      }
    }
    return x;
  }

  // Row-major operands, k-values 32 kb + 8 g .. of row spread(i, l15).
  static __device__ __forceinline__ uint32_t row_base(int l15, int g) { return at(spread(0, l15), 8 * g); }
  static __device__ __forceinline__ OP row(const char* lds, uint32_t base, int i, int kb) {
    const char* p = lds + 32 * (i >> 1) * kRow + ((base ^ (4 * (i & 1) * kRow)) ^ (64 * kb));
    OP f;
#pragma unroll
    for (int n = 0; n < kParts; ++n) f.p[n] = __builtin_bit_cast(bf8, *reinterpret_cast<const u4*>(p + n * kPart));
    return f;
  }
  // Transposed operands: k runs over the tile's rows 32 kb + 8 g .., and lane
  // l15 has column spread(i, l15). A group of 16 lanes reads 4 columns of 4
  // rows each and gets them transposed: lane l15 fetches row l15 / 4 of the
  // columns of lanes 4 (l15 % 4) ..
  static __device__ __forceinline__ uint32_t col_base(int l15, int g) {
    return at(8 * g + (l15 >> 2), spread(0, 4 * (l15 & 3)));
  }
  // What takes a column base from spread(0, .) to spread(i, .).
  static __device__ __forceinline__ uint32_t col_step(int i) { return (i >> 1) * 64 + (i & 1) * 8; }
  static __device__ __forceinline__ OP col(const char* lds, uint32_t base, int i, int kb) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4* lds_s4;
    const char* p = lds + 32 * kb * kRow + (base ^ col_step(i));
    OP f;
#pragma unroll
    for (int n = 0; n < kParts; ++n) {
      const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + n * kPart)));
      const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + n * kPart + 4 * kRow)));
      const u4 v = {lo.x, lo.y, hi.x, hi.y};
      f.p[n] = __builtin_bit_cast(bf8, v);
    }
    return f;
  }
};

// Where a workgroup works. Ids are dealt to the eight XCDs in turn; the
// workgroups that read the same q and k (the column slices and heads of one
// group, and the roles) follow one another on one XCD and share its L2.
__host__ __device__ __forceinline__ int slices(int vd) { return (vd + kVS - 1) / kVS; }
struct Place {
  int role, slice, b, h, seg;
  bool live;
};
__device__ __forceinline__ Place place(const LaArgs& a, int nseg) {
  const int id = blockIdx.x, rep = a.nheads / a.ngroups, sub = rep * a.nslices;
  const int j = id >> 3;
  int s = j % sub;
  const int unit = (j / sub) * 8 + (id & 7);
  Place p;
  p.live = unit < a.batch * a.ngroups * nseg;
  const int h = s / a.nslices;
  s -= h * a.nslices;
  p.role = 0;
  for (int n; p.role + 1 < a.nroles && s >= (n = slices(a.role[p.role].vd)); ++p.role) s -= n;
  p.slice = s;
  const int bg = unit / nseg;
  p.seg = unit - bg * nseg;
  p.b = bg / a.ngroups;
  p.h = (bg - p.b * a.ngroups) * rep + h;
  return p;
}

template <int KD>
__device__ __forceinline__ int64_t ws_base(const LaArgs& a, const Place& p, int seg) {
  const int64_t bh = (static_cast<int64_t>(p.role) * a.batch + p.b) * a.nheads + p.h;
  return ((bh * a.nseg + seg) * a.nsl + p.slice) * (KD * kVS);
}

// What a workgroup reads: the rows of one operand and head, from the first
// token on in the direction of the sum.
template <typename T>
__device__ __forceinline__ Rows rows_of(const LaOperand& o, const Place& pl, int rep, int width, int from, int most,
                                        int64_t first, bool rev) {
  const int64_t head = static_cast<int64_t>(o.per_group ? pl.h / rep : pl.h) * width + from;
  return Rows{reinterpret_cast<const char*>(static_cast<const T*>(o.p) + first * o.row + head),
              static_cast<uint32_t>(o.row * static_cast<int64_t>(sizeof(T))),
              static_cast<uint32_t>(min(width - from, most) * sizeof(T)), Order{rev}};
}

// The first tokens of documents among a chunk's 64, as bits (each wave asks
// for itself, a chunk ahead): a token whose id is not its predecessor's.
struct Ids {
  int own, prev;
  __device__ __forceinline__ void load(const int32_t* seq_idx, int64_t first, bool rev, int c, int seqlen, int lane) {
    // the 65 ids from the chunk's lowest token (forwards: the one before it) on
    const int pos = c * kC + lane;
    const int32_t* low = seq_idx + first + (rev ? -static_cast<int64_t>(c * kC + kC - 1) : c * kC - 1);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t*>(low), 0, (kC + 1) * 4, 0x00020000);
    const bool ok = (pos < seqlen) & (pos > 0);
    own = __builtin_amdgcn_raw_buffer_load_b32(rsrc, in_range(4 * (rev ? kC - 1 - lane : lane + 1), ok), 0, 0);
    prev = __builtin_amdgcn_raw_buffer_load_b32(rsrc, in_range(4 * (rev ? kC - lane : lane), ok), 0, 0);
  }
  __device__ __forceinline__ uint64_t begins() const { return __ballot(own != prev); }
};
// The last document's first token among those that begin in the chunk (0: none does).
__device__ __forceinline__ int last_of(uint64_t begins) { return begins ? 63 - __builtin_clzll(begins) : 0; }

// S^T of one wave: column v0 + spread(wave, l15), k-elements spread(i, 4 g) + r.
// Kernels and workspace hold half the state, which is exact, so that rounding its
// first part to bfloat16 takes no finite one to infinity.
constexpr float kHalf = 0.5f;
template <int KD>
struct State {
  static constexpr int kTiles = KD / 16;
  f4 t[kTiles];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) t[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // Half of one head's state [vd][kd] ([kd][vd] where `transposed`), zero beyond kd.
  __device__ __forceinline__ void load(const float* st, bool transposed, int col, int vd, int kd, int g) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int e = spread(i, 4 * g);
      if (e >= kd) continue;
      if (transposed) {
#pragma unroll
        for (int r = 0; r < 4; ++r) t[i][r] = st[static_cast<int64_t>(e + r) * vd + col];
      } else {
        t[i] = *reinterpret_cast<const f4*>(st + static_cast<int64_t>(col) * kd + e);
      }
      t[i] *= kHalf;
    }
  }
  // S^T = lam^n S^T + K^T (w V) over the tokens of the last document; w_in
  // holds the tokens' weights, keep is lam^n.
  //
  // The state is kept in float32, so for bfloat16 io as well the products w v (24
  // significant bits) are three parts. Two (`three` false) are left of them where
  // the state is never returned, in the sums for dq and dk, which read it in two
  // parts themselves (193 us instead of 201 for the gradients of 8 x 2048 tokens,
  // 12 heads of 128).
  template <int IO, bool SEQ, typename TileK>
  __device__ __forceinline__ void add(const char* Ks, uint32_t at_col, const Op<IO> (&vf)[2], const float* w_in,
                                      float keep, uint64_t begins, int g, int kd, bool three) {
    bool odd = false;  // a value is not finite
    const int last = SEQ ? last_of(begins) : 0;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) t[i][r] = SEQ && begins ? 0.0f : t[i][r] * keep;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float x[8];
      const f4 w[2] = {*reinterpret_cast<const f4*>(w_in + 32 * kb + 8 * g),
                       *reinterpret_cast<const f4*>(w_in + 32 * kb + 8 * g + 4)};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = get(vf[kb], j) * w[j >> 2][j & 3];
        if (SEQ) x[j] = 32 * kb + 8 * g + j >= last ? x[j] : 0.0f;
      }
      const u4 first = pack<false>(x);
      rest(x, first);
      if (IO == 1 && __any(unfit(first, 0.0f) != 0.0f)) {  // an infinity or NaN is whole in its first part: its rest is NaN
        asm volatile("");                                  // a branch, not selects
        odd = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] == x[j] ? x[j] : 0.0f;
      }
      // four tiles at a time: their operands first, then one product with each part in turn
      auto products = [&](const auto& parts) {
#pragma unroll
        for (int i0 = 0; i0 < kTiles; i0 += 4) {
          Op<IO> kf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) kf[i] = TileK::col(Ks, at_col, i0 + i, kb);
          // keys of other documents may hold infinities or NaN, which a weight of 0 would not remove
          if (SEQ && begins) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kf[i] = between(kf[i], last - (32 * kb + 8 * g), 7);
          }
          mma_each(t + i0, kf, parts);
        }
      };
      const u4 second = pack<false>(x);
      const bf8 p0 = __builtin_bit_cast(bf8, first), p1 = __builtin_bit_cast(bf8, second);
      if (IO == 0 || three) {
        rest(x, second);
        products(Parts<3>{{p0, p1, __builtin_bit_cast(bf8, pack<false>(x))}});
      } else {
        products(Parts<2>{{p0, p1}});
      }
    }
    if (IO == 1 && odd) {  // 0 again beyond kd, where the keys are 0
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        if (spread(i, 4 * g) >= kd) t[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }
};

// What lies in LDS: K, V and S twice each where they fit, then a chunk has one
// barrier; else K and V twice and S once, or each once, with a second barrier
// between the last reading of a chunk's and the writing of the next one's.
template <int IO, int KD>
struct Plan {
  static constexpr int kThreadsY = 2 * kThreads;
  using TileK = Tile<IO, KD, kThreadsY>;
  using TileV = Tile<IO, kVS, kThreadsY>;
  using TileS = Tile<IO, KD, kThreadsY, Sum<IO>>;  // [column of v][k-element]
  static constexpr int kKV = TileK::kBytes + TileV::kBytes, kS = TileS::kBytes, kMost = 160 * 1024 - 1024;
  static constexpr int kTBuf = 2 * kKV + kS <= kMost ? 2 : 1, kSBuf = 2 * kKV + 2 * kS <= kMost ? 2 : 1;
  static_assert(kTBuf * kKV + kSBuf * kS <= kMost, "LDS");
  // Chunks that K, V and Q are ahead in registers: two, but one where two would
  // spill (float32 128 wide: 8 x 2048, 12 heads, 178 us, 198 with two) and where
  // two workgroups share a CU and its registers (bfloat16 64 wide: 8 x 2048, 24
  // heads, packed: gradients 143 us, 174 with two; 130 and 129 us not packed).
  static constexpr int kAhead = (IO == 0) == (KD == 128) ? 1 : 2;
};

template <int IO, int KD, bool SEQ>
__global__ __launch_bounds__(2 * kThreads) __attribute__((amdgpu_waves_per_eu(IO == 1 ? 4 : 2))) void la_kernel(
    const LaArgs a) {
  using P = Plan<IO, KD>;
  using T = typename Io<IO>::T;
  using TileK = typename P::TileK;
  using TileV = typename P::TileV;
  using TileS = typename P::TileS;
  constexpr int kKb = KD / 32, kSum = IO == 1 ? 2 : 3, kTBuf = P::kTBuf, kSBuf = P::kSBuf, kAhead = P::kAhead;
  constexpr uint32_t kBufK = 0, kBufV = kTBuf * TileK::kBytes, kBufS = kBufV + kTBuf * TileV::kBytes;
  __shared__ __attribute__((aligned(512))) char lds[kBufS + kSBuf * TileS::kBytes];
  // powers of lam with their factors: of a score at distance 63 - m (0 from 64
  // on, above the diagonal), and of token s on its way into the state, for a
  // whole chunk and for the last one
  __shared__ float w_score[96], w_in[2][kC];

  const Place pl = place(a, a.nseg);
  if (!pl.live) return;
  const LaRole& R = a.role[pl.role];
  int kd = R.kd, vd = R.vd;
  const int v0 = pl.slice * kVS;
  // kept in scalar registers, not loaded again in the loop
  float sc_out = R.sc_out, sc_kv = R.sc_kv;
  void* out_p = R.out;
  int es_out = IO == 0 || R.out_f32 ? 4 : 2, off = R.off, rev_i = R.rev, nheads = a.nheads, seqlen = a.seqlen;
  int three_i = R.keeps;
  asm volatile("" : "+s"(sc_out), "+s"(sc_kv), "+s"(out_p), "+s"(es_out), "+s"(off), "+s"(rev_i), "+s"(nheads),
               "+s"(seqlen), "+s"(kd), "+s"(vd), "+s"(three_i));
  const bool rev = rev_i != 0, three = three_i != 0;
  const int tid = threadIdx.x, lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wv = wave & 3;
  const bool makes_y = wave < 4;
  const int rep = a.nheads / a.ngroups;
  const int nchunks = (seqlen + kC - 1) / kC;
  const int c0 = pl.seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nchunks);
  const float g2 = a.log_decay[pl.h] * kLog2e;
  const int64_t first = static_cast<int64_t>(pl.b) * seqlen + (rev ? seqlen - 1 : 0);
  const Rows qr = rows_of<T>(R.q, pl, rep, kd, 0, KD, first, rev), kr = rows_of<T>(R.k, pl, rep, kd, 0, KD, first, rev);
  const Rows vr = rows_of<T>(R.v, pl, rep, vd, v0, kVS, first, rev);

  const float keep_full = power(g2, kC);

  TileK kt[kAhead];
  TileV vt[kAhead];
  Ids ids[2];
  const typename TileK::Ways way_k(kr, tid);
  const typename TileV::Ways way_v(vr, tid);
  auto fetch = [&](int c, TileK& k, TileV& v) {
    const int n = c < c1 ? min(kC, seqlen - c * kC) : 0;
    k.load(kr, way_k, c, n);
    v.load(vr, way_v, c, n);
  };
  auto start = [&]() {
    fetch(c0, kt[0], vt[0]);
    if (kAhead == 2) fetch(c0 + 1, kt[kAhead - 1], vt[kAhead - 1]);
    if (SEQ) ids[0].load(a.seq_idx, first, rev, c0, seqlen, lane);
  };
  // A chunk's beginning, for either task: the tiles two chunks on start their
  // way, and the wave learns where documents begin.
  auto begin = [&](int c, auto parity) {
    constexpr int par = decltype(parity)::value;
    fetch(c + kAhead, kt[par % kAhead], vt[par % kAhead]);
    const uint64_t begins = SEQ ? ids[par].begins() : 0;
    if (SEQ) ids[par ^ 1].load(a.seq_idx, first, rev, c + 1, seqlen, lane);
    return begins;
  };
  auto put_tiles = [&](auto parity) {
    constexpr int par = decltype(parity)::value, buf = par % kTBuf;
    kt[par % kAhead].store(lds + kBufK + buf * TileK::kBytes, tid);
    vt[par % kAhead].store(lds + kBufV + buf * TileV::kBytes, tid);
  };
  // The two tasks run loops of their own, so that neither holds the other's
  // registers; they meet at the same number of barriers.
  auto all_chunks = [&](auto&& chunk) {
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    put_tiles(Even{});
    __syncthreads();
    for (int c = c0; c < c1; c += 2) {  // the second of the last two may be empty
      chunk(c, Even{});
      put_tiles(Odd{});
      __syncthreads();
      chunk(c + 1, Odd{});
      put_tiles(Even{});
      __syncthreads();
    }
  };

  if (!makes_y) {
    const int col = v0 + spread(wv, l15);
    State<KD> S;
    // writes this wave's columns of S to the chunk's tile
    auto put_state = [&](char* to) {
#pragma unroll
      for (int i = 0; i < State<KD>::kTiles; ++i) TileS::template put4<false>(to + TileS::at(spread(wv, l15), spread(i, 4 * g)), S.t[i]);
    };
    start();
    S.zero();
    if (a.nseg > 1) {
      // also segment 0, which has the join's copy of state_in: by now the last
      // segment may have written state_out in its place
      const float* w = a.ws + ws_base<KD>(a, pl, pl.seg);
#pragma unroll
      for (int i = 0; i < State<KD>::kTiles; ++i)
        S.t[i] = *reinterpret_cast<const f4*>(w + (i * kThreads + (tid & (kThreads - 1))) * 4);
    } else if (R.state_in && col < vd) {
      S.load(R.state_in + (static_cast<int64_t>(pl.b) * nheads + pl.h) * vd * kd, R.state_t, col, vd, kd, g);
    }
    put_state(lds + kBufS);
    if (wv < 2) {
      const int n = wv == 0 ? kC : seqlen - (nchunks - 1) * kC;
      w_in[wv][lane] = lane < n ? power(g2, n - off - lane) * (kHalf * sc_kv) : 0.0f;
    }
    const uint32_t col_k = TileK::col_base(l15, g);
    const uint32_t col_v = TileV::col_base(l15, g) ^ TileV::col_step(wv);
    all_chunks([&](int c, auto parity) {
      constexpr int par = decltype(parity)::value;
      const int n = min(kC, seqlen - c * kC);
      const uint64_t begins = begin(c, parity);
      uint32_t at_col = col_k, at_v = col_v;  // renewed: what follows from them is not kept over the loop
      int gg = g;
      asm volatile("" : "+v"(at_col), "+v"(at_v), "+v"(gg));
      if (c < c1) {
        Op<IO> vf[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) vf[kb] = TileV::col(lds + kBufV + par % kTBuf * TileV::kBytes, at_v, 0, kb);
        const float keep = n == kC ? keep_full : power(g2, n);
        const char* Ks = lds + kBufK + par % kTBuf * TileK::kBytes;
        S.template add<IO, SEQ, TileK>(Ks, at_col, vf, w_in[n < kC], keep, begins, gg, kd, three);
      }
      if (kSBuf == 1) __syncthreads();  // the chunk's starting state has been read
      put_state(lds + kBufS + (kSBuf == 2 ? par ^ 1 : 0) * TileS::kBytes);
    });
    if (c1 == nchunks && R.state_out && col < vd) {
      float* st = R.state_out + (static_cast<int64_t>(pl.b) * nheads + pl.h) * vd * kd + static_cast<int64_t>(col) * kd;
#pragma unroll
      for (int i = 0; i < State<KD>::kTiles; ++i) {
        const int e = spread(i, 4 * g);
        if (e < kd) *reinterpret_cast<f4*>(st + e) = S.t[i] * (1.0f / kHalf);
      }
    }
    return;
  }

  // the wave's 16 tokens of q as operands; 0 beyond the sequence and beyond kd
  constexpr int kQ = sizeof(T) / 2;  // 16-byte pieces of 8 elements
  u4 q[kAhead][kKb][kQ];
  uint32_t way_q[kKb];
#pragma unroll
  for (int kb = 0; kb < kKb; ++kb)
    way_q[kb] = in_range(qr.order.far(16 * wv + l15) * qr.stride + (32 * kb + 8 * g) * sizeof(T), 32 * kb + 8 * g < kd);
  auto fetch_q = [&](int c, u4 (&f)[kKb][kQ]) {
    const int n = c < c1 ? min(kC, seqlen - c * kC) : 0;
    const auto rsrc = qr.chunk(c, n);
    const uint32_t cut = qr.order.cut(n) * qr.stride;
#pragma unroll
    for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
      for (int i = 0; i < kQ; ++i)
        f[kb][i] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, way_q[kb] - cut, 16 * i, 0));
  };
  start();
  fetch_q(c0, q[0]);
  if (kAhead == 2) fetch_q(c0 + 1, q[kAhead - 1]);
  if (tid < 96) w_score[tid] = tid < kC ? power(g2, 63 - tid) * (sc_out * sc_kv) : 0.0f;
  const float w_out = power(g2, 16 * wv + l15 + off) * (sc_out / kHalf);  // of the state read at this lane's token
  const int64_t out_row = static_cast<int64_t>(nheads) * vd;
  const Rows outs{static_cast<char*>(out_p) + (first * out_row + static_cast<int64_t>(pl.h) * vd + v0) * es_out,
                  static_cast<uint32_t>(out_row * es_out), static_cast<uint32_t>(min(vd - v0, kVS) * es_out), Order{rev}};
  uint32_t way_out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    way_out[h] = in_range(outs.order.far(16 * wv + l15) * outs.stride + (32 * h + 8 * g) * es_out, 32 * h + 8 * g < vd - v0);
  const uint32_t row_b = TileK::row_base(l15, g), col_v = TileV::col_base(l15, g);
  all_chunks([&](int c, auto parity) {
    constexpr int par = decltype(parity)::value;
    const int n = c < c1 ? min(kC, seqlen - c * kC) : 0;
    const char* const Ks = lds + kBufK + par % kTBuf * TileK::kBytes;
    const char* const Vs = lds + kBufV + par % kTBuf * TileV::kBytes;
    const char* const Ss = lds + kBufS + (kSBuf == 2 ? par : 0) * TileS::kBytes;
    const uint64_t begins = begin(c, parity);
    uint32_t at_row = row_b, at_v = col_v;  // renewed: what follows from them is not kept over the loop
    int t = 16 * wv + l15, gg = g;
    asm volatile("" : "+v"(at_row), "+v"(at_v), "+v"(t), "+v"(gg));
    int from = 0;      // where token t's document begins in the chunk
    bool open = true;  // no document begins between the state and token t
    if (SEQ) {
      const uint64_t m = begins & (~0ull >> (63 - t));
      from = last_of(m);
      open = m == 0;
    }
    Op<IO> qf[kKb];
#pragma unroll
    for (int kb = 0; kb < kKb; ++kb) {
      if constexpr (IO == 1) {
        qf[kb] = Op<1>{{__builtin_bit_cast(bf8, q[par % kAhead][kb][0])}};
      } else {
        const f4 lo = __builtin_bit_cast(f4, q[par % kAhead][kb][0]), hi = __builtin_bit_cast(f4, q[par % kAhead][kb][kQ - 1]);
        qf[kb] = split<3>(lo, hi);
      }
    }
    if (kAhead == 1) fetch_q(c + 1, q[0]);  // what it held is in the operands
    f4 y[4];  // columns t, rows spread(i, 4 g) + r of the 64 columns of v
    if (c < c1) {
      // the scores: columns t, rows s; tiles 0 and 1 have s < 32, the other two are needed by the upper 32 tokens
      f4 sc[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sc[2 * h] = sc[2 * h + 1] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        if (h == 1 && wv < 2) break;
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) {
          const Op<IO> kf[2] = {TileK::row(Ks, at_row, 2 * h, kb), TileK::row(Ks, at_row, 2 * h + 1, kb)};
          mma_each(sc + 2 * h, kf, qf[kb]);
        }
#pragma unroll
        for (int i = 2 * h; i < 2 * h + 2; ++i) {
          const int s = spread(i, 4 * gg);
          const float* w = w_score + 63 - t + s;
          const f4 wt = {w[0], w[1], w[2], w[3]};
#pragma unroll
          for (int r = 0; r < 4; ++r)  // later tokens have weight 0, those of other documents are dropped
            sc[i][r] = !SEQ || s + r >= from ? sc[i][r] * wt[r] : 0.0f;
        }
      }
      // rows of S's tiles at a time: four would spill in 128 registers (8 x 2048,
      // 24 heads of 64, packed: gradients 150 us with four, 147 with two)
      constexpr int kG = IO == 1 && KD == 64 ? 2 : 4;
      auto carried = [&](uint32_t at, auto again) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) {
#pragma unroll
          for (int i0 = 0; i0 < 4; i0 += kG) {
            Sum<IO> sf[kG];
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              sf[i] = TileS::row(Ss, at, i0 + i, kb);
              if (again.value) sf[i] = whole(sf[i]);
            }
            mma_each(y + i0, sf, qf[kb]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[i][r] = open ? y[i][r] * w_out : 0.0f;
      };
      carried(at_row, std::false_type{});
      const Sum<IO> s0 = tiles_op<kSum>(sc[0], sc[1], gg), s1 = tiles_op<kSum>(sc[2], sc[3], gg);
      auto weighted = [&](const Sum<IO>& p, int kb) {
        Op<IO> vf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[i] = TileV::col(Vs, at_v, i, kb);
        mma_each(y, vf, p);
      };
      weighted(s0, 0);
      if (wv >= 2) weighted(s1, 1);
      float bad = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) bad = fmaf(y[i][r], 0.0f, bad);
      // An infinity or NaN in k or v also reaches the tokens that it is masked
      // for, as 0 * inf. Where any sum is not finite the sums are taken again, in
      // the same order, with 0 for masked scores, for values that are not finite
      // and for the rests of scores and states that are not; the values are added
      // behind, where they are not masked. So a sum that none of them belongs to
      // has the bits that it has without them.
      if (__any(bad != 0.0f)) {
        uint32_t again = row_b, again_v = col_v;
        asm volatile("" : "+v"(again), "+v"(again_v));  // read again, not kept from above
        carried(again, std::true_type{});
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const int o = 32 * kb + 8 * gg;  // token of the lane's first score
          const Sum<IO> p = whole(between(kb == 0 ? s0 : s1, from - o, t - o));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Op<IO> v = TileV::col(Vs, again_v, i, kb), vf[1] = {masked(v, finite(v))};
            mma_each(y + i, vf, p);
          }
#pragma unroll 1
          for (int gs = 0; gs < 4; ++gs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int s = 32 * kb + 8 * gs + j;
              const float w = __shfl(get(p, j), 16 * gs + l15, 64);
              if (s > t || s < from) continue;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const f4 v = TileV::get4(Vs, s, spread(i, 4 * gg));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (v[r] * 0.0f != 0.0f) y[i][r] = fmaf(w, v[r], y[i][r]);
              }
            }
          }
        }
      }
    }
    if (kSBuf == 1) __syncthreads();  // the chunk's starting state has been read
    if (kAhead == 2) fetch_q(c + 2, q[par % kAhead]);
    // Two tiles are 8 neighbouring columns of a token, the upper four first
    // where g is odd. Rows from n on and columns from vd on are out of the
    // buffer's range and dropped.
    const auto rsrc = outs.chunk(c, n);
    const uint32_t cut = outs.order.cut(n) * outs.stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = way_out[h] - cut;
      if (IO == 0 || es_out == 4) {
        const bool up = gg & 1;
        const f4 lo = up ? y[2 * h + 1] : y[2 * h], hi = up ? y[2 * h] : y[2 * h + 1];
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, lo), rsrc, o, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, hi), rsrc, o + 16, 0, 0);
      } else {
        const Op<1> v = tiles_op<1>(y[2 * h], y[2 * h + 1], gg);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v.p[0]), rsrc, o, 0, 0);
      }
    }
  });
}

// What each segment but the last adds to the state: the state's task alone,
// four waves to a workgroup and two or three workgroups to a CU, so that one
// chunk ahead suffices (1 x 65536, 12 heads of 128, bfloat16: 390 MB in 105 us,
// 3.7 TB/s; 131 us with two chunks ahead, which spilled).
template <int IO, int KD, bool SEQ>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(IO == 1 ? 3 : 2))) void la_sum_kernel(
    const LaArgs a) {
  using T = typename Io<IO>::T;
  using TileK = Tile<IO, KD, kThreads>;
  using TileV = Tile<IO, kVS, kThreads>;
  constexpr uint32_t kBufV = TileK::kBytes;
  __shared__ __attribute__((aligned(512))) char lds[kBufV + TileV::kBytes];
  __shared__ float w_in[kC];

  const Place pl = place(a, a.nseg - 1);
  if (!pl.live) return;
  const LaRole& R = a.role[pl.role];
  const int kd = R.kd, vd = R.vd, v0 = pl.slice * kVS, seqlen = a.seqlen;
  const bool rev = R.rev;
  const int tid = threadIdx.x, lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rep = a.nheads / a.ngroups;
  const int seg0 = pl.seg * a.seg_chunks, c1 = seg0 + a.seg_chunks;  // whole chunks: a later segment follows
  const float g2 = a.log_decay[pl.h] * kLog2e;
  const int64_t first = static_cast<int64_t>(pl.b) * seqlen + (rev ? seqlen - 1 : 0);
  const Rows kr = rows_of<T>(R.k, pl, rep, kd, 0, KD, first, rev);
  const Rows vr = rows_of<T>(R.v, pl, rep, vd, v0, kVS, first, rev);
  const bool three = R.keeps;
  // Only the segment's last document adds to its state: the sum starts in the
  // chunk where that begins, found from the segment's end, 1024 tokens at a time
  // (2 x 4133, 24 heads of 64 x 96, float32: 30 us for all sums, 44 in full).
  int c0 = seg0;
  bool seen = false;  // a document begins in this segment
  if (SEQ) {
    __shared__ int newest[2][kThreads / 64];
    const int32_t* ids = a.seq_idx + first;
    const int sign = rev ? -1 : 1;
    for (int end = c1 * kC, half = 0; end > seg0 * kC && !seen; end -= 4 * kThreads, half ^= 1) {
      int at = -1;
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const int pos = end - 1 - i * kThreads - tid;
        if (pos >= seg0 * kC && pos > 0)
          at = max(at, ids[sign * static_cast<int64_t>(pos)] != ids[sign * static_cast<int64_t>(pos - 1)] ? pos : -1);
      }
      for (int o = 32; o > 0; o >>= 1) at = max(at, __shfl_xor(at, o, 64));
      if (lane == 0) newest[half][wv] = at;
      __syncthreads();
      at = max(max(newest[half][0], newest[half][1]), max(newest[half][2], newest[half][3]));
      seen = at >= 0;
      if (seen) c0 = at / kC;
    }
    c0 = __builtin_amdgcn_readfirstlane(c0);
  }

  TileK kt;
  TileV vt;
  Ids marks;
  const typename TileK::Ways way_k(kr, tid);
  const typename TileV::Ways way_v(vr, tid);
  auto fetch = [&](int c) {
    const int n = c < c1 ? kC : 0;
    kt.load(kr, way_k, c, n);
    vt.load(vr, way_v, c, n);
  };
  fetch(c0);
  if (SEQ) marks.load(a.seq_idx, first, rev, c0, seqlen, lane);
  if (tid < kC) w_in[tid] = power(g2, kC - R.off - tid) * (kHalf * R.sc_kv);
  const float keep = power(g2, kC);
  State<KD> S;
  S.zero();
  kt.store(lds, tid);
  vt.store(lds + kBufV, tid);
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    fetch(c + 1);
    const uint64_t begins = SEQ ? marks.begins() : 0;
    if (SEQ) marks.load(a.seq_idx, first, rev, c + 1, seqlen, lane);
    uint32_t at_col = TileK::col_base(l15, g), at_v = TileV::col_base(l15, g) ^ TileV::col_step(wv);
    asm volatile("" : "+v"(at_col), "+v"(at_v));  // renewed, as in la_kernel
    Op<IO> vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) vf[kb] = TileV::col(lds + kBufV, at_v, 0, kb);
    S.template add<IO, SEQ, TileK>(lds, at_col, vf, w_in, keep, begins, g, kd, three);
    __syncthreads();
    kt.store(lds, tid);
    vt.store(lds + kBufV, tid);
    __syncthreads();
  }
  float* w = a.ws + ws_base<KD>(a, pl, pl.seg + 1);
#pragma unroll
  for (int i = 0; i < State<KD>::kTiles; ++i) *reinterpret_cast<f4*>(w + (i * kThreads + tid) * 4) = S.t[i];
  // every head and slice of the row writes the same value
  if (SEQ && tid == 0) a.flags[(pl.role * a.batch + pl.b) * a.nseg + pl.seg] = seen ? 1 : 0;
}

// The state before each segment: entry 0 is the incoming state, and entry j,
// which holds the sum of segment j - 1 alone, becomes lam^len entry (j - 1) +
// entry j. One thread per 4 elements, in the order in which State keeps them.
template <int KD, bool SEQ>
__global__ __launch_bounds__(kThreads) void la_join_kernel(const LaArgs a) {
  constexpr int kTiles = KD / 16;
  const int i = blockIdx.x % kTiles;
  int rest = blockIdx.x / kTiles;
  Place p;
  p.slice = rest % a.nsl;
  rest /= a.nsl;
  p.role = rest % a.nroles;
  rest /= a.nroles;
  p.h = rest % a.nheads;
  p.b = rest / a.nheads;
  const LaRole& R = a.role[p.role];
  if (p.slice * kVS >= R.vd) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int col = p.slice * kVS + spread(tid >> 6, lane & 15), e = spread(i, 4 * (lane >> 4));
  f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (R.state_in && col < R.vd && e < R.kd) {
    const float* st = R.state_in + (static_cast<int64_t>(p.b) * a.nheads + p.h) * R.vd * R.kd;
    if (R.state_t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] = st[static_cast<int64_t>(e + r) * R.vd + col];
    } else {
      s = *reinterpret_cast<const f4*>(st + static_cast<int64_t>(col) * R.kd + e);
    }
    s *= kHalf;
  }
  const float g2 = a.log_decay[p.h] * kLog2e, keep = power(g2, a.seg_chunks * kC);
  float* w = a.ws + ws_base<KD>(a, p, 0) + (i * kThreads + tid) * 4;
  const int64_t step = static_cast<int64_t>(a.nsl) * KD * kVS;
  *reinterpret_cast<f4*>(w) = s;
  for (int j = 1; j < a.nseg; ++j) {
    const bool cut = SEQ && a.flags[(p.role * a.batch + p.b) * a.nseg + j - 1] != 0;
    const f4 own = *reinterpret_cast<const f4*>(w + j * step);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // over a long segment keep is 0 or infinite where lam is neither: a state of
      // 0 stays 0, and an infinite one infinite
      const bool as_is = s[r] == 0.0f || (__builtin_isinf(s[r]) && g2 > -HUGE_VALF);
      s[r] = cut ? own[r] : as_is ? s[r] + own[r] : fmaf(s[r], keep, own[r]);
    }
    *reinterpret_cast<f4*>(w + j * step) = s;
  }
}

template <int IO, int KD, bool SEQ>
hipError_t launch_typed(const LaCall& c, const LaPlan& p, const LaArgs& a) {
  const int64_t sub = static_cast<int64_t>(a.nheads / a.ngroups) * a.nslices;
  auto grid = [&](int nseg) {
    const int64_t units = static_cast<int64_t>(a.batch) * a.ngroups * nseg;
    return dim3(static_cast<unsigned>((units + 7) / 8 * 8 * sub));
  };
  if (p.nseg > 1) {
    hipLaunchKernelGGL((la_sum_kernel<IO, KD, SEQ>), grid(p.nseg - 1), dim3(kThreads), 0, c.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned joins = static_cast<unsigned>(KD / 16) * a.nsl * a.nroles * a.nheads * a.batch;
    hipLaunchKernelGGL((la_join_kernel<KD, SEQ>), dim3(joins), dim3(kThreads), 0, c.stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((la_kernel<IO, KD, SEQ>), grid(p.nseg), dim3(2 * kThreads), 0, c.stream, a);
  return hipGetLastError();
}

int padded(int32_t d) { return d <= 64 ? 64 : 128; }

size_t state_floats(const LaPlan& p, int32_t batch, int32_t nheads, int32_t kd, int32_t vd, int32_t nroles) {
  return static_cast<size_t>(nroles) * batch * nheads * p.nseg * slices(vd) * padded(kd) * kVS;
}

}  // namespace

// The estimate counts one workgroup on a CU: the sums of a call run in rounds of
// 32 workgroups on each XCD, and segments fill the rounds where sequences are
// few. (Of bfloat16 heads of up to 64 two fit, which hide one another's waits
// rather than halve the time. Counted as two, without the second parts of scores
// and state: 8 x 2048, 24 heads, 65 us instead of 43, the gradients of 4 x 4096,
// 16 heads, 90 instead of 75; only 1 x 65536, 12 heads, gained, 135 instead of
// 145.)
// Splitting reads k and v once more: the number of segments with the least
// estimated time is taken, in chunks of one workgroup. A workgroup costs two
// beside its own, a chunk of the segment sums 0.6 (they are as long as the
// segment, or as all of them take at the rate of a CU), the join 2 and an eighth
// for each segment. Measured: 8 x 2048, 12 heads of 128, bf16, 192 workgroups,
// 73 us in one segment, 106 in four; 1 x 65536, 24 workgroups, 355 us in 21
// segments, 358 in 32, 368 in 10; 2 x 4133, 24 heads of 64 x 96, float32, packed,
// 96 workgroups, 131 us in 5, 148 in 8, 130 in 2 (144, 155 and 180 while the sums
// read whole segments, as without documents).
LaPlan la_plan(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v, int32_t nroles) {
  const int32_t nchunks = (seqlen + kC - 1) / kC;
  const int64_t units = static_cast<int64_t>(batch) * ngroups;
  // a backward call makes d_k columns twice and d_v columns once
  const int64_t sub = static_cast<int64_t>(nheads / ngroups) * (nroles == 1 ? slices(d_v) : 2 * slices(d_k) + slices(d_v));
  // workgroups of the fullest CU
  auto load = [&](int64_t nseg) { return static_cast<double>((units * nseg + 7) / 8 * sub) / 32; };
  LaPlan best{1, nchunks};
  double least = 0;
  for (int32_t n = 1; n <= 256 && (n == 1 || n <= nchunks / 4); ++n) {
    const int32_t len = (nchunks + n - 1) / n;
    if (n > 1 && (nchunks + len - 1) / len != n) continue;  // as many segments as a smaller n
    double t = std::ceil(load(n)) * (len + 2);
    if (n > 1) t += 2 + n / 8.0 + 0.6 * len * std::max(load(n - 1), 1.0);
    if (n == 1 || t < least) {
      least = t;
      best.nseg = n;
      best.seg_chunks = len;
    }
  }
  return best;
}

size_t la_ws_floats(const LaPlan& p, int32_t batch, int32_t nheads, int32_t d_k, int32_t d_v, int32_t nroles) {
  if (p.nseg <= 1) return 0;
  const int32_t most = d_k > d_v ? d_k : d_v;  // the roles of a backward call exchange the two
  const size_t flags = (static_cast<size_t>(nroles) * batch * p.nseg + 63) / 64 * 64;
  return flags + state_floats(p, batch, nheads, nroles > 1 ? most : d_k, nroles > 1 ? most : d_v, nroles);
}

hipError_t launch_la(const LaCall& c, const LaPlan& p) {
  LaArgs a{};
  a.batch = c.batch;
  a.seqlen = c.seqlen;
  a.nheads = c.nheads;
  a.ngroups = c.ngroups;
  a.nseg = p.nseg;
  a.seg_chunks = p.seg_chunks;
  a.nroles = c.nroles;
  a.seq_idx = c.seq_idx;
  a.log_decay = c.log_decay;
  int kd = 0, vd = 0;
  for (int r = 0; r < c.nroles; ++r) {
    a.role[r] = c.role[r];
    kd = kd > c.role[r].kd ? kd : c.role[r].kd;
    vd = vd > c.role[r].vd ? vd : c.role[r].vd;
  }
  a.nsl = slices(vd);
  for (int r = 0; r < c.nroles; ++r) a.nslices += slices(c.role[r].vd);
  a.flags = reinterpret_cast<int32_t*>(c.workspace);
  a.ws = c.workspace + (static_cast<size_t>(c.nroles) * c.batch * p.nseg + 63) / 64 * 64;
  const bool wide = padded(kd) == 128;
  if (c.io_dtype == 0) {
    if (c.seq_idx) return wide ? launch_typed<0, 128, true>(c, p, a) : launch_typed<0, 64, true>(c, p, a);
    return wide ? launch_typed<0, 128, false>(c, p, a) : launch_typed<0, 64, false>(c, p, a);
  }
  if (c.seq_idx) return wide ? launch_typed<1, 128, true>(c, p, a) : launch_typed<1, 64, true>(c, p, a);
  return wide ? launch_typed<1, 128, false>(c, p, a) : launch_typed<1, 64, false>(c, p, a);
}

namespace {

template <int IO>
__global__ __launch_bounds__(kThreads) void la_head_sum_kernel(int64_t n, int32_t rep, int32_t d4,
                                                              const float* __restrict__ part,
                                                              typename Io<IO>::T* __restrict__ out) {
  // one thread per 4 outputs; n = rows * groups * d / 4
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t rg = i / d4;
    const float* p = part + (rg * rep * d4 + (i - rg * d4)) * 4;
    f4 s = *reinterpret_cast<const f4*>(p);
    for (int h = 1; h < rep; ++h) s += *reinterpret_cast<const f4*>(p + static_cast<int64_t>(h) * d4 * 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) Io<IO>::store(out + i * 4 + r, s[r]);
  }
}

// One token. A state row (one column of v) is spread over LN lanes of 4
// k-elements each; the kernel reads and writes the state once and is bound by
// that traffic (256 conversations, 12 heads of 128: 406 MB in 70 us, 5.8 TB/s,
// above the rate of a large copy, for part of it stays in the last-level cache).
template <int IO, int LN>
__global__ __launch_bounds__(kThreads) void la_step_kernel(const LaStepCall a, int64_t rows) {
  using T = typename Io<IO>::T;
  const int64_t gid = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = gid / LN;
  const int e = static_cast<int>(threadIdx.x % LN) * 4;
  const bool live = row < rows && e < a.d_k;
  const int64_t r = row < rows ? row : rows - 1;  // idle lanes mirror the last row and store nothing
  const int64_t bh = r / a.d_v;
  const int j = static_cast<int>(r - bh * a.d_v);
  const int b = static_cast<int>(bh / a.nheads), h = static_cast<int>(bh - static_cast<int64_t>(b) * a.nheads);
  const int grp = h / (a.nheads / a.ngroups);
  const float g2 = a.log_decay[h] * kLog2e;
  float part = 0.0f;
  if (live) {
    const float lam = exp2_hw(g2);
    const float v = Io<IO>::load(static_cast<const T*>(a.v) + b * a.v_row + static_cast<int64_t>(h) * a.d_v + j);
    const T* k = static_cast<const T*>(a.k) + b * a.k_row + static_cast<int64_t>(grp) * a.d_k + e;
    const T* q = static_cast<const T*>(a.q) + b * a.q_row + static_cast<int64_t>(grp) * a.d_k + e;
    const f4 s0 = __builtin_nontemporal_load(reinterpret_cast<const f4*>(a.state_in + r * a.d_k + e));
    f4 s1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s1[i] = fmaf(lam, s0[i], v * Io<IO>::load(k + i));
      part = fmaf(Io<IO>::load(q + i), s1[i], part);
    }
    __builtin_nontemporal_store(s1, reinterpret_cast<f4*>(a.state_out + r * a.d_k + e));
  }
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) part += __shfl_xor(part, o, LN);
  if (live && e == 0) Io<IO>::store(static_cast<T*>(a.y) + r, part * a.scale);
}

template <int IO, int LN>
hipError_t launch_step_typed(const LaStepCall& c) {
  const int64_t rows = static_cast<int64_t>(c.batch) * c.nheads * c.d_v;
  const int64_t blocks = (rows * LN + kThreads - 1) / kThreads;
  const int64_t gx = blocks < (int64_t{1} << 22) ? blocks : (int64_t{1} << 22);
  hipLaunchKernelGGL((la_step_kernel<IO, LN>),
                     dim3(static_cast<unsigned>(gx), static_cast<unsigned>((blocks + gx - 1) / gx)), dim3(kThreads), 0,
                     c.stream, c, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_la_head_sum(int64_t rows, int32_t nheads, int32_t ngroups, int32_t d, int32_t io_dtype,
                              const float* part, void* out, hipStream_t stream) {
  const int64_t n = rows * ngroups * (d / 4), blocks = (n + kThreads - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(blocks < 65536 ? blocks : 65536));
  if (io_dtype == 0)
    hipLaunchKernelGGL(la_head_sum_kernel<0>, grid, dim3(kThreads), 0, stream, n, nheads / ngroups, d / 4, part,
                       static_cast<float*>(out));
  else
    hipLaunchKernelGGL(la_head_sum_kernel<1>, grid, dim3(kThreads), 0, stream, n, nheads / ngroups, d / 4, part,
                       static_cast<uint16_t*>(out));
  return hipGetLastError();
}

hipError_t launch_la_step(const LaStepCall& c) {
  if (c.io_dtype == 0) {
    if (c.d_k <= 32) return launch_step_typed<0, 8>(c);
    return c.d_k <= 64 ? launch_step_typed<0, 16>(c) : launch_step_typed<0, 32>(c);
  }
  if (c.d_k <= 32) return launch_step_typed<1, 8>(c);
  return c.d_k <= 64 ? launch_step_typed<1, 16>(c) : launch_step_typed<1, 32>(c);
}

}  // namespace mscan
