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
// A workgroup of four waves walks the chunks of one (batch row, head, 64
// columns of v) in order. A wave keeps the state of its 16 columns in
// accumulators, S^T tiles [16 k-elements x 16 columns], from the first chunk
// to the last. A^T = K Q^T goes through LDS (each wave makes up to three of
// the ten 16x16 tiles on and below the diagonal); y^T = V^T A^T + S Q^T and
// S^T += K^T (w V) follow, V^T and K^T read transposed from row-major tiles.
// The rows of the S^T tiles are numbered (`spread`) so that the accumulators a
// lane holds of two tiles are 8 consecutive k-elements: the A operand of S Q^T
// as they stand.
#include "linattn_internal.h"
#include "mfma_frag.h"
#include "scan_device.h"

namespace mscan {

namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kVS = 64;        // columns of v per workgroup
constexpr int kThreads = 256;  // four waves of 16 columns
constexpr int kMaxRoles = 3;

struct LaArgs {
  int32_t batch, seqlen, nheads, ngroups, nseg, seg_chunks, nroles, nsl;
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

// Element j of a fragment as float32.
__device__ __forceinline__ float frag_get(const Frag<1>& f, int j) { return static_cast<float>(f.v[j]); }
__device__ __forceinline__ float frag_get(const Frag<0>& f, int j) { return j < 4 ? f.lo[j & 3] : f.hi[j & 3]; }

// Zero the k-values of a lane's eight that lie below `first`.
__device__ __forceinline__ Frag<1> frag_from(const Frag<1>& f, int first) {
  u4 v = __builtin_bit_cast(u4, f.v);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] &= (2 * j >= first ? 0xFFFFu : 0u) | (2 * j + 1 >= first ? 0xFFFF0000u : 0u);
  return Frag<1>{__builtin_bit_cast(bf8, v)};
}
__device__ __forceinline__ Frag<0> frag_from(const Frag<0>& f, int first) {
  Frag<0> r = f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < first) r.lo[j] = 0.0f;
    if (4 + j < first) r.hi[j] = 0.0f;
  }
  return r;
}

// The A operand of S Q^T from two neighbouring S^T tiles: 8 consecutive
// k-elements, of which the first tile has the upper four where g is odd.
template <int IO>
__device__ __forceinline__ Frag<IO> state_frag(f4 even, f4 odd, int g);
template <>
__device__ __forceinline__ Frag<1> state_frag<1>(f4 even, f4 odd, int g) {
  const u4 v = __builtin_bit_cast(u4, frag_regs<1>(even, odd).v);
  const bool up = g & 1;
  const u4 w = {up ? v.z : v.x, up ? v.w : v.y, up ? v.x : v.z, up ? v.y : v.w};
  return Frag<1>{__builtin_bit_cast(bf8, w)};
}
template <>
__device__ __forceinline__ Frag<0> state_frag<0>(f4 even, f4 odd, int g) {
  return g & 1 ? Frag<0>{odd, even} : Frag<0>{even, odd};
}

// The weighted values w V as matrix-core operands. The state is kept and
// returned in float32, so for bfloat16 io the products w v (24 significant
// bits) are split into bfloat16 parts, each the rounded rest of those before
// it, and multiplied once for each: three parts hold all 24 bits. Where the
// state is not returned, only y sees it, rounded to bfloat16 itself, and two
// parts (16 bits) do; one would double the rounding that y gets.
template <int IO>
struct Weighted;
template <>
struct Weighted<1> {
  static constexpr int kParts = 3;
  Frag<1> part[3];
  __device__ __forceinline__ void set(const float (&x)[8], bool three) {
    float r[8], bad = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = x[j];
      bad = fmaf(x[j], 0.0f, bad);
    }
    const bool inf = __any(bad != 0.0f);  // an infinity or NaN is whole in its first part
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      if (p == 2 && !three) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __bf16 h = static_cast<__bf16>(r[j]);
        part[p].v[j] = h;
        r[j] -= static_cast<float>(h);
      }
      if (inf) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = r[j] == r[j] ? r[j] : 0.0f;
      }
    }
  }
};
template <>
struct Weighted<0> {
  static constexpr int kParts = 1;
  Frag<0> part[1];
  __device__ __forceinline__ void set(const float (&x)[8], bool) {
    part[0] = Frag<0>{f4{x[0], x[1], x[2], x[3]}, f4{x[4], x[5], x[6], x[7]}};
  }
};

// The column (of a tile, or of the state) that row or column m of a wave's i-th
// 16-wide product stands for. Two neighbouring i share 32 columns: m / 4 = c
// has columns 8 c .. 8 c + 3 of them in one and 8 c + 4 .. 8 c + 7 in the other,
// the lower four first for even c (so that one transposed read takes both
// halves of the 16-byte pieces, and with them all banks).
__device__ __forceinline__ int spread(int i, int m) {
  const int c = m >> 2;
  return 32 * (i >> 1) + 8 * c + 4 * ((i ^ c) & 1) + (m & 3);
}

// A 64-row tile of W columns in LDS and its way there from global memory
// through registers (the load is issued a chunk ahead).
//
// The 16-byte pieces of a row are exchanged by an exclusive-or with a number
// made of the row's low bits, so that each way of reading hits every bank
// once: 16 rows of one piece (operands with k along the row), and, in half a
// wave of transposed reads, rows 0-3 and 8-11 of four half pieces.
//
// All reads are (base ^ constant) + constant with a base that depends on the
// lane alone: a step along the row changes bits that the exchange leaves to
// the exclusive-or, and 16 rows further the exchange is the same.
template <int IO, int W>
struct Tile {
  using T = typename Io<IO>::T;
  static constexpr uint32_t kRow = W * sizeof(T);  // bytes
  static constexpr uint32_t kBytes = kC * kRow;
  static constexpr int kPer = kRow / 16;
  static constexpr int kN = kC * kPer / kThreads;
  u4 v[kN];

  static __device__ __forceinline__ uint32_t exchange(int row) {
    // 8 pieces a row: two rows span the banks, so the row's lowest bit is left
    // out; else its low four bits, the middle two swapped
    return kPer == 8 ? (row >> 1) & 7 : (row & 9) | ((row & 2) << 1) | ((row & 4) >> 1);
  }
  static __device__ __forceinline__ uint32_t at(int row, int byte) {
    return static_cast<uint32_t>(row) * kRow + (static_cast<uint32_t>(byte) ^ (exchange(row) << 4));
  }
  // Rows 0 .. n - 1 of the chunk, row r at p + r * step (step in bytes, of either
  // sign); rows from n on and columns from `cols` on are zero: the buffer
  // range's answer to an offset out of range.
  __device__ __forceinline__ void load(const void* p, int64_t step, int n, int cols, int tid) {
    const uint32_t stride = static_cast<uint32_t>(step < 0 ? -step : step), width = min(cols, W) * sizeof(T);
    const char* low = static_cast<const char*>(p) + (step < 0 ? step * (n - 1) : 0);
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(low), 0,
                                                        stride * static_cast<uint32_t>(n - 1) + width, 0x00020000);
    // a thread's pieces lie in one column, kThreads / kPer rows apart
    asm volatile("" : "+v"(tid));  // the offsets are cheaper made again than kept over the loop
    const uint32_t c = static_cast<uint32_t>(tid % kPer) * 16;
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int r = tid / kPer + q * (kThreads / kPer);
      const uint32_t off = static_cast<uint32_t>(step < 0 ? n - 1 - r : r) * stride + c;
      v[q] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, r < n && c < width ? off : 0xFFFFFFF0u, 0, 0));
    }
  }
  __device__ __forceinline__ void store(char* lds, int tid) const {
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int i = tid + q * kThreads, r = i / kPer;
      *reinterpret_cast<u4*>(lds + at(r, (i - r * kPer) * 16)) = v[q];
    }
  }

  // Row-major operands, k-values 32 kb + 8 g .. of row 16 i + l15.
  static __device__ __forceinline__ uint32_t row_base(int l15, int g) { return at(l15, 8 * g * sizeof(T)); }
  static __device__ __forceinline__ Frag<IO> row(const char* lds, uint32_t base, int i, int kb) {
    const char* p = lds + 16 * i * kRow;
    const uint32_t a = base ^ (32 * kb * sizeof(T));
    if constexpr (IO == 1) {
      return Frag<1>{__builtin_bit_cast(bf8, *reinterpret_cast<const u4*>(p + a))};
    } else {
      return Frag<0>{*reinterpret_cast<const f4*>(p + a), *reinterpret_cast<const f4*>(p + (a ^ 16))};
    }
  }
  // Transposed operands: k runs over the tile's rows 32 kb + 8 g .., and lane
  // l15 has column spread(i, l15).
  static __device__ __forceinline__ uint32_t col_base(int l15, int g) {
    // bfloat16: a group of 16 lanes reads 4 columns of 4 rows each and gets
    // them transposed: lane l15 fetches row l15 / 4 of the columns of lanes 4 (l15 % 4) ..
    if constexpr (IO == 1) return at(8 * g + (l15 >> 2), spread(0, 4 * (l15 & 3)) * 2);
    return at(8 * g, spread(0, l15) * 4);
  }
  static __device__ __forceinline__ Frag<IO> col(const char* lds, uint32_t base, int i, int kb) {
    const uint32_t a = base ^ (((i >> 1) * 32 + (i & 1) * 4) * sizeof(T));  // spread(i, .) is spread(0, .) ^ this
    const char* p = lds + 32 * kb * kRow;
    if constexpr (IO == 1) {
      typedef short s4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s4* lds_s4;
      const uint32_t x4 = (exchange(4) << 4);  // rows 4 to 7 of the eight
      const u2 lo = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + a)));
      const u2 hi = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + 4 * kRow + (a ^ x4))));
      const u4 v = {lo.x, lo.y, hi.x, hi.y};
      return Frag<1>{__builtin_bit_cast(bf8, v)};
    } else {
      Frag<0> f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f.lo[j] = *reinterpret_cast<const float*>(p + j * kRow + (a ^ (exchange(j) << 4)));
        f.hi[j] = *reinterpret_cast<const float*>(p + (4 + j) * kRow + (a ^ (exchange(4 + j) << 4)));
      }
      return f;
    }
  }
};

// Where a workgroup works. Ids are dealt to the eight XCDs in turn; the
// workgroups that read the same q and k (the column slices and heads of one
// group, and the roles) follow one another on one XCD and share its L2.
struct Place {
  int role, slice, b, h, seg;
  bool live;
};
__device__ __forceinline__ Place place(const LaArgs& a, int nseg) {
  const int id = blockIdx.x, rep = a.nheads / a.ngroups, sub = a.nroles * rep * a.nsl;
  const int j = id >> 3;
  int s = j % sub;
  const int unit = (j / sub) * 8 + (id & 7);
  Place p;
  p.live = unit < a.batch * a.ngroups * nseg;
  p.role = s % a.nroles;
  s /= a.nroles;
  p.slice = s % a.nsl;
  const int bg = unit / nseg;
  p.seg = unit - bg * nseg;
  p.b = bg / a.ngroups;
  p.h = (bg - p.b * a.ngroups) * rep + s / a.nsl;
  return p;
}

template <int KD>
__device__ __forceinline__ int64_t ws_base(const LaArgs& a, const Place& p, int seg) {
  const int64_t bh = (static_cast<int64_t>(p.role) * a.batch + p.b) * a.nheads + p.h;
  return ((bh * a.nseg + seg) * a.nsl + p.slice) * (KD * kVS);
}

// STATE: only the sum that a segment adds to the state (segments 0 .. nseg - 2).
template <int IO, int KD, bool SEQ, bool STATE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(IO == 1 ? 3 : KD == 64 ? 2 : 1))) void la_kernel(
    const LaArgs a) {
  using T = typename Io<IO>::T;
  using TileK = Tile<IO, KD>;
  using TileV = Tile<IO, kVS>;
  using TileA = Tile<IO, kC>;
  constexpr int kTiles = KD / 16, kKb = KD / 32;
  __shared__ __attribute__((aligned(512))) char lds[(STATE ? 1 : 2) * TileK::kBytes + (STATE ? 1 : 2) * TileV::kBytes];
  char* const Ks = lds;
  char* const Vs = lds + TileK::kBytes;
  char* const As = Vs + TileV::kBytes;  // [t][s]
  char* const Qs = As + TileA::kBytes;
  // powers of lam with their factors: of a score at distance 63 - m (0 from 64 on, above the diagonal), of the
  // state read at token t, of token s on its way into the state of a chunk of n
  __shared__ float w_score[80], w_out[kC], w_in[kC];

  const Place pl = place(a, STATE ? a.nseg - 1 : a.nseg);
  if (!pl.live) return;
  const LaRole& R = a.role[pl.role];
  int kd = R.kd, vd = R.vd;
  const int v0 = pl.slice * kVS;
  if (v0 >= vd) return;
  // kept in scalar registers, not loaded again in the loop
  float sc_out = R.sc_out, sc_kv = R.sc_kv;
  void* out_p = R.out;
  const bool three = R.state_out != nullptr;
  int es_out = IO == 0 || R.out_f32 ? 4 : 2, off = R.off, rev_i = R.rev, nheads = a.nheads, seqlen = a.seqlen;
  asm volatile("" : "+s"(sc_out), "+s"(sc_kv), "+s"(out_p), "+s"(es_out), "+s"(off), "+s"(rev_i), "+s"(nheads),
               "+s"(seqlen), "+s"(kd), "+s"(vd));
  const bool rev = rev_i != 0;
  const int tid = threadIdx.x, lane = tid & 63, l15_ = lane & 15, g_ = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rep = a.nheads / a.ngroups, grp = pl.h / rep;
  const int nchunks = (a.seqlen + kC - 1) / kC;
  const int c0 = pl.seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, nchunks);
  const float g2 = a.log_decay[pl.h] * kLog2e;
  const int64_t row0 = static_cast<int64_t>(pl.b) * a.seqlen;

  const int64_t first = row0 + (rev ? a.seqlen - 1 : 0);
  const int64_t es = rev ? -static_cast<int64_t>(sizeof(T)) : static_cast<int64_t>(sizeof(T));
  const int64_t qs = R.q.row * es, ks = R.k.row * es, vs = R.v.row * es;  // bytes from a token to the next one
  const T* qp = static_cast<const T*>(R.q.p) + first * R.q.row + static_cast<int64_t>(R.q.per_group ? grp : pl.h) * kd;
  const T* kp = static_cast<const T*>(R.k.p) + first * R.k.row + static_cast<int64_t>(R.k.per_group ? grp : pl.h) * kd;
  const T* vp = static_cast<const T*>(R.v.p) + first * R.v.row + static_cast<int64_t>(R.v.per_group ? grp : pl.h) * vd + v0;

  // the state of this lane: column v0 + spread(wv, l15), k-elements spread(i, 4 g) + r
  const int col = v0 + spread(wv, l15_);
  f4 S[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) S[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  if (!STATE) {
    if (a.nseg > 1) {
      // also segment 0, which has the join's copy of state_in: by now the last
      // segment may have written state_out in its place
      const float* w = a.ws + ws_base<KD>(a, pl, pl.seg);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) S[i] = *reinterpret_cast<const f4*>(w + (i * kThreads + tid) * 4);
    } else if (R.state_in && col < vd) {
      const float* st = R.state_in + (static_cast<int64_t>(pl.b) * a.nheads + pl.h) * vd * kd;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int e = spread(i, 4 * g_);
        if (e >= kd) continue;
        if (R.state_t) {
#pragma unroll
          for (int r = 0; r < 4; ++r) S[i][r] = st[static_cast<int64_t>(e + r) * vd + col];
        } else {
          S[i] = *reinterpret_cast<const f4*>(st + static_cast<int64_t>(col) * kd + e);
        }
      }
    }
    // the two 16x16 tiles above the diagonal that the products read
    for (int i = tid; i < 512; i += kThreads) {
      const int t = i >> 8, r = (i >> 4) & 15, c = i & 15;
      Io<IO>::store(reinterpret_cast<T*>(As + TileA::at(32 * t + r, (32 * t + 16 + c) * sizeof(T))), 0.0f);
    }
  }

  if (!STATE && tid < 80) w_score[tid] = tid < kC ? power(g2, 63 - tid) * (sc_out * sc_kv) : 0.0f;
  if (!STATE && tid < kC) w_out[tid] = power(g2, tid + off) * sc_out;
  const float keep_full = power(g2, kC);

  TileK kt, qt;
  TileV vt;
  int id_own = 0, id_prev = 0;
  bool seen = false;  // a document began in this segment
  auto fetch = [&](int c) {
    const int rows = min(kC, seqlen - c * kC);
    auto from = [&](const T* p, int64_t step) {
      return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + static_cast<int64_t>(c) * kC * step);
    };
    kt.load(from(kp, ks), ks, rows, kd, tid);
    vt.load(from(vp, vs), vs, rows, vd - v0, tid);
    if (!STATE) qt.load(from(qp, qs), qs, rows, kd, tid);
    if (SEQ) {
      const int pos = c * kC + lane;
      id_own = id_prev = 0;
      if (pos < seqlen && pos > 0) {
        id_own = a.seq_idx[first + (rev ? -pos : pos)];
        id_prev = a.seq_idx[first + (rev ? 1 - pos : pos - 1)];
      }
    }
  };
  fetch(c0);

  const uint32_t row_b = TileK::row_base(l15_, g_), col_b = TileK::col_base(l15_, g_);
  const uint32_t a_b = TileA::row_base(l15_, g_), v_b = TileV::col_base(l15_, g_);
  for (int c = c0; c < c1; ++c) {
    // Renewed in each chunk: the addresses that follow from these would
    // otherwise all be kept in registers over the whole loop.
    uint32_t at_row = row_b, at_col = col_b, at_a = a_b, at_v = v_b;
    int l15 = l15_, g = g_;
    asm volatile("" : "+v"(at_row), "+v"(at_col), "+v"(at_a), "+v"(at_v), "+v"(l15), "+v"(g));
    const int n = min(kC, seqlen - c * kC);
    kt.store(Ks, tid);
    vt.store(Vs, tid);
    if (!STATE) qt.store(Qs, tid);
    if ((c == c0 || n < kC) && tid < kC) w_in[tid] = tid < n ? power(g2, n - off - tid) * sc_kv : 0.0f;
    // bit s: a document begins at token s of the chunk
    const uint64_t begins = SEQ ? __ballot(id_own != id_prev) : 0;
    const int last = begins ? 63 - __builtin_clzll(begins) : 0;  // the last document's first token
    seen |= begins != 0;
    __syncthreads();
    if (c + 1 < c1) fetch(c + 1);

    if (!STATE) {
      // A^T: rows s, columns t; wave j has the 16 tokens t from 16 j on, and each lane 4 rows s of one column t
      const int j = wv, t = 16 * j + l15;
      int from = 0;
      if (SEQ) {
        const uint64_t m = begins & (~0ull >> (63 - t));
        from = m ? 63 - __builtin_clzll(m) : 0;
      }
      const char* q_at = Qs + 16 * j * TileK::kRow;
      char* a_at = As + 16 * j * TileA::kRow;
      const uint32_t to = TileA::at(l15, 4 * g * sizeof(T));
      Frag<IO> qf[kKb], kf[kKb];
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb) {
        kf[kb] = TileK::row(Ks, at_row, 0, kb);
        qf[kb] = TileK::row(q_at, at_row, 0, kb);
      }
#pragma unroll 1
      for (int i = 0; i <= j; ++i) {
        f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) acc = mma(kf[kb], qf[kb], acc);
        const int s = 16 * i + 4 * g;
        const float* w = w_score + 63 - t + s;
        const f4 wt = {w[0], w[1], w[2], w[3]};
        if (i < j) {
#pragma unroll
          for (int kb = 0; kb < kKb; ++kb) kf[kb] = TileK::row(Ks + 16 * (i + 1) * TileK::kRow, at_row, 0, kb);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)  // chosen, not multiplied, so that masked pairs drop infinities and NaN
          acc[r] = s + r <= t && s + r >= from ? acc[r] * wt[r] : 0.0f;
        char* dst = a_at + (to ^ (16 * i * sizeof(T)));  // row t, from column s
        if (IO == 1) {
          typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
          const bf4 v = {static_cast<__bf16>(acc[0]), static_cast<__bf16>(acc[1]), static_cast<__bf16>(acc[2]),
                         static_cast<__bf16>(acc[3])};
          *reinterpret_cast<u2*>(dst) = __builtin_bit_cast(u2, v);
        } else {
          *reinterpret_cast<f4*>(dst) = acc;
        }
      }
      __syncthreads();
    }

    Frag<IO> vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) vf[kb] = TileV::col(Vs, at_v, wv, kb);

    if (!STATE) {
      f4 y[4];
      // the state's part, lam^(t + off) S q_t; `from[j]`: where token t's document begins in the chunk
      int from[4];
      auto carried = [&](uint32_t at) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) {
          Frag<IO> qf[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) qf[j] = TileK::row(Qs, at, j, kb);
          const Frag<IO> sf = state_frag<IO>(S[2 * kb], S[2 * kb + 1], g);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = mma(sf, qf[j], y[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 16 * j + l15;
          from[j] = 0;
          bool open = true;  // no document begins between the state and token t
          if (SEQ) {
            const uint64_t m = begins & (~0ull >> (63 - t));
            from[j] = m ? 63 - __builtin_clzll(m) : 0;
            open = m == 0;
          }
          const float w = w_out[t];
#pragma unroll
          for (int r = 0; r < 4; ++r) y[j][r] = open ? y[j][r] * w : 0.0f;
        }
      };
      carried(at_row);
      float bad = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = mma(vf[0], TileA::row(As, at_a, j, 0), y[j]);
        if (j >= 2) y[j] = mma(vf[1], TileA::row(As, at_a, j, 1), y[j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) bad = fmaf(y[j][r], 0.0f, bad);
      }
      // An infinity or NaN in v also reaches the tokens that it is masked for,
      // as 0 * inf. Where any sum is not finite the sums are taken again, over
      // the unmasked tokens alone.
      if (__any(bad != 0.0f)) {
        uint32_t again = at_row;
        asm volatile("" : "+v"(again));  // read again, not kept from above
        carried(again);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 16 * j + l15;
#pragma unroll 1
          for (int s = 0; s < kC; ++s) {
            if (s > t || s < from[j]) continue;
            const float p = Io<IO>::load(reinterpret_cast<const T*>(As + TileA::at(t, s * sizeof(T))));
            const T* v = reinterpret_cast<const T*>(Vs + TileV::at(s, spread(wv, 4 * g) * sizeof(T)));
#pragma unroll
            for (int r = 0; r < 4; ++r) y[j][r] = fmaf(p, Io<IO>::load(v + r), y[j][r]);
          }
        }
      }
      // each lane holds 4 consecutive columns of one token; rows from n on and
      // columns from vd on are out of the buffer's range and dropped
      const int oc = spread(wv, 4 * g);
      const uint32_t row_out = static_cast<uint32_t>(nheads) * vd * es_out;
      const int64_t low = first + (rev ? -static_cast<int64_t>(c * kC + n - 1) : c * kC);
      char* const out = static_cast<char*>(out_p) + ((low * nheads + pl.h) * vd + v0) * es_out;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(out, 0, row_out * (n - 1) + (vd - v0) * es_out, 0x00020000);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 16 * j + l15;
        const uint32_t o = t < n && oc < vd - v0
                               ? static_cast<uint32_t>(rev ? n - 1 - t : t) * row_out + static_cast<uint32_t>(oc) * es_out
                               : 0xFFFFFFF0u;
        if (IO == 0 || es_out == 4) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, y[j]), rsrc, o, 0, 0);
        } else {
          typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
          const bf4 v = {static_cast<__bf16>(y[j][0]), static_cast<__bf16>(y[j][1]), static_cast<__bf16>(y[j][2]),
                         static_cast<__bf16>(y[j][3])};
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), rsrc, o, 0, 0);
        }
      }
    }

    // S^T = lam^n S^T + K^T (w V) over the tokens of the last document
    const float keep = n == kC ? keep_full : power(g2, n);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = begins ? 0.0f : S[i][r] * keep;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      float x[8];
      const f4 w[2] = {*reinterpret_cast<const f4*>(w_in + 32 * kb + 8 * g),
                       *reinterpret_cast<const f4*>(w_in + 32 * kb + 8 * g + 4)};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = frag_get(vf[kb], j) * w[j >> 2][j & 3];
        if (SEQ) x[j] = 32 * kb + 8 * g + j >= last ? x[j] : 0.0f;
      }
      Weighted<IO> wvf;
      wvf.set(x, three);
      // four tiles at a time: their operands first, then one product with each part in turn
#pragma unroll
      for (int i0 = 0; i0 < kTiles; i0 += 4) {
        Frag<IO> kf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          kf[i] = TileK::col(Ks, at_col, i0 + i, kb);
          if (SEQ) kf[i] = frag_from(kf[i], last - (32 * kb + 8 * g));
        }
#pragma unroll
        for (int p = Weighted<IO>::kParts - 1; p >= 0; --p) {
          if (p == 2 && !three) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) S[i0 + i] = mma(kf[i], wvf.part[p], S[i0 + i]);
        }
      }
    }
    __syncthreads();
  }

  if (STATE) {
    float* w = a.ws + ws_base<KD>(a, pl, pl.seg + 1);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) *reinterpret_cast<f4*>(w + (i * kThreads + tid) * 4) = S[i];
    if (SEQ && tid == 0) {
      // every head and slice of the row writes the same value
      a.flags[(pl.role * a.batch + pl.b) * a.nseg + pl.seg] = seen ? 1 : 0;
    }
  } else if (c1 == nchunks && R.state_out && col < vd) {
    float* st = R.state_out + (static_cast<int64_t>(pl.b) * a.nheads + pl.h) * vd * kd + static_cast<int64_t>(col) * kd;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int e = spread(i, 4 * g_);
      if (e < kd) *reinterpret_cast<f4*>(st + e) = S[i];
    }
  }
}

// The state before each segment: entry 0 is the incoming state, and entry j,
// which holds the sum of segment j - 1 alone, becomes lam^len entry (j - 1) +
// entry j. One thread per 4 elements, in the order in which la_kernel keeps them.
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
  }
  const float keep = power(a.log_decay[p.h] * kLog2e, a.seg_chunks * kC);
  float* w = a.ws + ws_base<KD>(a, p, 0) + (i * kThreads + tid) * 4;
  const int64_t step = static_cast<int64_t>(a.nsl) * KD * kVS;
  *reinterpret_cast<f4*>(w) = s;
  for (int j = 1; j < a.nseg; ++j) {
    const bool cut = SEQ && a.flags[(p.role * a.batch + p.b) * a.nseg + j - 1] != 0;
    const f4 own = *reinterpret_cast<const f4*>(w + j * step);
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = cut ? own[r] : fmaf(s[r], keep, own[r]);
    *reinterpret_cast<f4*>(w + j * step) = s;
  }
}

template <int IO, int KD, bool SEQ>
hipError_t launch_typed(const LaCall& c, const LaPlan& p, const LaArgs& a) {
  const int64_t sub = static_cast<int64_t>(a.nroles) * (a.nheads / a.ngroups) * a.nsl;
  auto grid = [&](int nseg) {
    const int64_t units = static_cast<int64_t>(a.batch) * a.ngroups * nseg;
    return dim3(static_cast<unsigned>((units + 7) / 8 * 8 * sub));
  };
  if (p.nseg > 1) {
    hipLaunchKernelGGL((la_kernel<IO, KD, SEQ, true>), grid(p.nseg - 1), dim3(kThreads), 0, c.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned joins = static_cast<unsigned>(KD / 16) * a.nsl * a.nroles * a.nheads * a.batch;
    hipLaunchKernelGGL((la_join_kernel<KD, SEQ>), dim3(joins), dim3(kThreads), 0, c.stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((la_kernel<IO, KD, SEQ, false>), grid(p.nseg), dim3(kThreads), 0, c.stream, a);
  return hipGetLastError();
}

int padded(int32_t d) { return d <= 64 ? 64 : 128; }

size_t state_floats(const LaPlan& p, int32_t batch, int32_t nheads, int32_t kd, int32_t vd, int32_t nroles) {
  const size_t nsl = (vd + kVS - 1) / kVS;
  return static_cast<size_t>(nroles) * batch * nheads * p.nseg * nsl * padded(kd) * kVS;
}

}  // namespace

LaPlan la_plan(int32_t batch, int32_t seqlen, int32_t nheads, int32_t d_k, int32_t d_v, int32_t nroles) {
  const int32_t nchunks = (seqlen + kC - 1) / kC;
  const int64_t groups = static_cast<int64_t>(nroles) * batch * nheads * ((d_v + kVS - 1) / kVS);
  const int64_t want = (512 + groups - 1) / groups, most = nchunks / 4 > 1 ? nchunks / 4 : 1;
  const int32_t nseg = static_cast<int32_t>(want < most ? want : most);
  LaPlan p;
  p.seg_chunks = (nchunks + nseg - 1) / nseg;
  p.nseg = (nchunks + p.seg_chunks - 1) / p.seg_chunks;
  return p;
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
  a.nsl = (vd + kVS - 1) / kVS;
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
// that traffic.
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
