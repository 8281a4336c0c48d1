// Gated delta rule on gfx950: what its kernels share.
//
// Per head, with a_t = sigmoid(gate_t) or exp(gate_t) and eta_t = lr_max sigmoid(beta_t + b):
//   e_t = v_t - a_t S_{t-1}^T k_t;  S_t = a_t S_{t-1} + eta_t k_t e_t^T;  o_t = scale S_t^T q_t.
// A chunk of C tokens that starts from the state S, with G_i = sum_{j<=i} log a_j and
// R_ij = e^{G_i - G_j}, has its updates u_i = eta_i e_i from one triangular system:
//   (1 + A) U = eta (V - e^G K S),  A_ij = eta_i R_ij k_i.k_j  (j < i);
//   O = scale (e^G Q S + (R o Q K^T) U);   S' = e^{G_C} S + K^T (e^{G_C - G} U).
// T = (1 + A)^-1 and the scores P = scale R o Q K^T do not depend on the state: one kernel
// forms them for every chunk at once, and only the products with S are walked through.
// Columns of S do not meet, so a wave walks 16 of them with no other wave's help.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mfma_util.h"
#include "ttt_device.h"
#include "ttt_internal.h"

namespace ttt {
namespace delta {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct Args {
  int B, T, H, Hk, dk, dv, dvp;  // dvp: dv rounded up to 32, the width of U, Y and the kept states
  int packed, gate_kind;
  int wide_q, wide_k, wide_v, wide_o, wide_do, wide_dv;  // whether every row of a head starts on 16 bytes
  int dense;                     // both q and k are wide: the walks read them where they are
  float scale, lr_max, lr_bias;
  int64_t n;                     // tokens
  int64_t ldq, ldk, ldv, ldg, ldb;
  int chunks, chunks_per_seq;    // chunk slots; of a sequence (dense)
  int nseg, seg_chunks;          // dense: the pieces that a sequence is walked in at the same time; a piece's chunks
  const float* seg_states;       // [B * nseg][H][dk][dv]: the states that enter them, where nseg > 1
  const int* base;               // packed: [B + 1] the sequences' first chunks
  const int4* table;             // packed: [chunks] first token, tokens, sequence
  const int* order;              // packed: [B] the sequences, the longest first
  const void* q;
  const void* k;
  const void* v;
  const void* gate;
  const void* beta;
  const float* s0;
  void* o;
  float* s_final;
  float* vec;                    // [chunks][H][3][C]: e^G, e^{G_C - G}, eta
  void* kq;                      // else [chunks][Hk][2][C][dkp]: keys and queries, padded with zeros
  char* t;                       // [chunks][H] T, or its transpose, in operand order
  char* p;                       // the same of the scores
  void* u;                       // [chunks][H][dvp][C], tokens in operand order (see token_col), in terms (see keep)
  void* before;                  // [chunks][H][dvp][dkp]: the state that enters the chunk, in terms
  void* y;                       // as u: T^T dU
  void* after;                   // as before: the gradient of the state that leaves it
  const void* d_o;
  const float* d_sfinal;
  void* dq;
  void* dk_out;
  void* dv_out;
  void* dgate;
  void* dbeta;
  float* ds0;
};

// Tokens of a chunk.  64 bf16 rows of 128 are 16 KB; fp32 rows are twice that, and the
// 256-channel backward keeps four such tiles in LDS.
template <typename E> struct Chunk;
template <> struct Chunk<bf16_t> { static constexpr int C = 64; };
template <> struct Chunk<float> { static constexpr int C = 32; };

struct Where {
  int64_t token;  // first
  int len, seq;
};

// A chunk's tokens; len < 0: the slot is empty.
template <int C> __device__ __forceinline__ Where locate(const Args& a, int chunk) {
  if (a.packed) {
    const int4 w = a.table[chunk];
    return {__builtin_amdgcn_readfirstlane(w.x), __builtin_amdgcn_readfirstlane(w.y), __builtin_amdgcn_readfirstlane(w.z)};
  }
  const int seq = chunk / a.chunks_per_seq, c = chunk % a.chunks_per_seq;
  return {static_cast<int64_t>(seq) * a.T + c * C, min(C, a.T - c * C), seq};
}

// ---- tiles in LDS ----

// A [rows][NCOL] tile: bf16 with swizzled 16-byte granules, fp32 with rows 16 bytes longer.
template <typename E, int NCOL> struct Tile;
template <int NCOL> struct Tile<bf16_t, NCOL> {
  static_assert(NCOL >= 32);
  static constexpr int kRow = NCOL;
  static __device__ __forceinline__ int at(int row, int col) { return swz<NCOL>(row, col); }
};
template <int NCOL> struct Tile<float, NCOL> {
  static constexpr int kRow = NCOL + 4;
  static __device__ __forceinline__ int at(int row, int col) { return row * kRow + col; }
};

// Rows 0 .. len - 1 and columns 0 .. nc - 1 of a row-major matrix into a tile of ROWS x NCOL; the
// rest becomes zero.  wide: every row starts on 16 bytes and nc is a whole number of pieces.
template <typename E, int ROWS, int NCOL, int THREADS>
__device__ __forceinline__ void stage(E* lds, const E* src, int64_t ld, int len, int nc, bool wide, int width = NCOL) {
  constexpr int V = 16 / sizeof(E);
  if (wide) {
    const int pieces = width / V;
    for (int i = threadIdx.x; i < ROWS * pieces; i += THREADS) {
      const int row = i / pieces, col = (i % pieces) * V;
      uint4 x = {0, 0, 0, 0};
      if (row < len && col < nc) x = *reinterpret_cast<const uint4*>(src + row * ld + col);
      *reinterpret_cast<uint4*>(lds + Tile<E, NCOL>::at(row, col)) = x;
    }
  } else {
    for (int i = threadIdx.x; i < ROWS * width; i += THREADS) {
      const int row = i / width, col = i % width;
      lds[Tile<E, NCOL>::at(row, col)] = row < len && col < nc ? src[row * ld + col] : E{};
    }
  }
}

// ---- matrix-core operands ----
//
// v_mfma_f32_16x16x32_bf16 and, for fp32, eight v_mfma_f32_16x16x4_f32: lane (i, g) = (l % 16,
// l / 16) of an A operand holds eight k of row i, of a B operand eight k of column i; which
// eight is free as long as A and B agree.  A result lane holds rows 4 g + r of column i, so two
// result tiles, one above the other, are a B operand whose k are {4 g + 0..3, 16 + 4 g + 0..3}.
// fp32 values that a bf16 product needs whole go in as two terms, x = hi + lo (2^-17 of x is lost).

template <typename E> struct Frag;
template <> struct Frag<bf16_t> { using Raw = bf16x8_t; };
struct f32x8 { f32x4_t a, b; };
template <> struct Frag<float> { using Raw = f32x8; };

template <typename E> struct Split;  // eight fp32 values as an operand
template <> struct Split<bf16_t> {
  bf16x8_t hi, lo;
  __device__ __forceinline__ Split() {}
  __device__ __forceinline__ Split(f32x4_t x, f32x4_t y) {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    u32x4_t h, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // two at a time: three vector instructions a value
      const float a = j < 2 ? x[2 * j] : y[2 * j - 4], b = j < 2 ? x[2 * j + 1] : y[2 * j - 3];
      h[j] = pack_bf16x2(a, b);
      l[j] = pack_bf16x2(a - __uint_as_float(h[j] << 16), b - __uint_as_float(h[j] & 0xffff0000u));
    }
    hi = __builtin_bit_cast(bf16x8_t, h);
    lo = __builtin_bit_cast(bf16x8_t, l);
  }
};
template <> struct Split<float> {
  f32x4_t a, b;
  __device__ __forceinline__ Split() {}
  __device__ __forceinline__ Split(f32x4_t x, f32x4_t y) : a(x), b(y) {}
};

// The same values in three terms (2^-25 is lost): what is added to a state, and the right-hand sides that it comes from.
// In two, the state was 3.6e-6 off and not fp32's 1e-7; the state in K S and T, in two terms, leave it 5e-7 off (128
// channels; 1e-6 to 3e-6 below 32).
template <typename E> struct Whole;
template <> struct Whole<bf16_t> {
  bf16x8_t hi, mid, lo;
  __device__ __forceinline__ Whole() {}
  __device__ __forceinline__ Whole(f32x4_t x, f32x4_t y) {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    u32x4_t h, m, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = j < 2 ? x[2 * j] : y[2 * j - 4], b = j < 2 ? x[2 * j + 1] : y[2 * j - 3];
      h[j] = pack_bf16x2(a, b);
      a -= __uint_as_float(h[j] << 16);
      b -= __uint_as_float(h[j] & 0xffff0000u);
      m[j] = pack_bf16x2(a, b);
      l[j] = pack_bf16x2(a - __uint_as_float(m[j] << 16), b - __uint_as_float(m[j] & 0xffff0000u));
    }
    hi = __builtin_bit_cast(bf16x8_t, h);
    mid = __builtin_bit_cast(bf16x8_t, m);
    lo = __builtin_bit_cast(bf16x8_t, l);
  }
};
template <> struct Whole<float> : Split<float> {
  using Split<float>::Split;
};

// A split's two 16-byte parts.
__device__ __forceinline__ bf16x8_t first_half(const Split<bf16_t>& s) { return s.hi; }
__device__ __forceinline__ bf16x8_t second_half(const Split<bf16_t>& s) { return s.lo; }
__device__ __forceinline__ f32x4_t first_half(const Split<float>& s) { return s.a; }
__device__ __forceinline__ f32x4_t second_half(const Split<float>& s) { return s.b; }
__device__ __forceinline__ void set_halves(Split<bf16_t>& s, bf16x8_t a, bf16x8_t b) { s.hi = a; s.lo = b; }
__device__ __forceinline__ void set_halves(Split<float>& s, f32x4_t a, f32x4_t b) { s.a = a; s.b = b; }

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4_t mma(f32x8 a, f32x8 b, f32x4_t c) { return mfma16(a.b, b.b, mfma16(a.a, b.a, c)); }
__device__ __forceinline__ f32x4_t mma(bf16x8_t a, bf16x8_t b, f32x4_t c) { return mfma16(a, b, c); }
// the first in two terms, the second exact in its type
__device__ __forceinline__ f32x4_t mma(const Split<bf16_t>& a, bf16x8_t b, f32x4_t c) { return mfma16(a.hi, b, mfma16(a.lo, b, c)); }
__device__ __forceinline__ f32x4_t mma(const Split<float>& a, f32x8 b, f32x4_t c) { return mfma16(a.b, b.b, mfma16(a.a, b.a, c)); }
// both in two terms
__device__ __forceinline__ f32x4_t mma(const Split<bf16_t>& a, const Split<bf16_t>& b, f32x4_t c) {
  return mfma16(a.hi, b.hi, mfma16(a.hi, b.lo, mfma16(a.lo, b.hi, c)));
}
__device__ __forceinline__ f32x4_t mma(const Split<float>& a, const Split<float>& b, f32x4_t c) {
  return mfma16(a.b, b.b, mfma16(a.a, b.a, c));
}
__device__ __forceinline__ f32x4_t zero4() { return f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}; }

// Eight consecutive columns of a row of a tile.
template <int NCOL> __device__ __forceinline__ bf16x8_t row_frag(const bf16_t* lds, int row, int col) {
  return *reinterpret_cast<const bf16x8_t*>(lds + Tile<bf16_t, NCOL>::at(row, col));
}
template <int NCOL> __device__ __forceinline__ f32x8 row_frag(const float* lds, int row, int col) {
  const float* p = lds + Tile<float, NCOL>::at(row, col);
  return {*reinterpret_cast<const f32x4_t*>(p), *reinterpret_cast<const f32x4_t*>(p + 4)};
}
// Rows r0 .. r0 + 3 and r1 .. r1 + 3 of a column.  Lane i's column is col4(i / 4) + i % 4, where
// col4 is what the lane i' with i' % 4 = i / 4 gave as `piece`: ds_read_b64_tr_b16 hands lane
// 4 a + b of each 16 lanes element b of the 8-byte pieces that lanes a, a + 4, a + 8, a + 12 name.
template <int NCOL>
__device__ __forceinline__ bf16x8_t col_frag(const bf16_t* lds, int r0, int r1, int piece, int /*col*/, int tid) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const int i4 = (tid & 15) >> 2;
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + Tile<bf16_t, NCOL>::at(r0 + i4, piece)));
  const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + Tile<bf16_t, NCOL>::at(r1 + i4, piece)));
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s z = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8_t, z);
}
template <int NCOL>
__device__ __forceinline__ f32x8 col_frag(const float* lds, int r0, int r1, int /*piece*/, int col, int /*tid*/) {
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.a[j] = lds[Tile<float, NCOL>::at(r0 + j, col)];
    f.b[j] = lds[Tile<float, NCOL>::at(r1 + j, col)];
  }
  return f;
}

// The states' tiles: row 4 g + r of tile t is channel 32 (t / 2) + 8 g + 4 (t % 2) + r, so a pair of
// tiles as a B operand has eight consecutive channels a lane.
__device__ __forceinline__ int state_row(int t, int g) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); }
// Column operand of tile t's rows over the tokens of a pair of token tiles (row 0 = token `tok`).
template <int NCOL, typename E>
__device__ __forceinline__ typename Frag<E>::Raw state_col(const E* lds, int tok, int t, int tid = threadIdx.x) {
  const int i = tid & 15, g = (tid & 63) >> 4;
  return col_frag<NCOL>(lds, tok + 4 * g, tok + 16 + 4 * g, state_row(t, i & 3), state_row(t, i >> 2) + (i & 3), tid);
}
// Column operand of columns col0 + i over rows row0 + 8 g + 0..7.
template <int NCOL, typename E>
__device__ __forceinline__ typename Frag<E>::Raw plain_col(const E* lds, int row0, int col0, int tid = threadIdx.x) {
  const int i = tid & 15, g = (tid & 63) >> 4;
  return col_frag<NCOL>(lds, row0 + 8 * g, row0 + 8 * g + 4, col0 + 4 * (i & 3), col0 + i, tid);
}

// U and Y are kept as [column][C] with the tokens of a pair of tiles in the order of the operand that they
// were: 8 g + j is token 4 g + j, or for j >= 4 token 16 + 4 g + j - 4.  This is the operand of token tile mt
// over 32 columns (rows), in the tokens' own order.
template <int NCOL, typename E>
__device__ __forceinline__ typename Frag<E>::Raw token_col(const E* lds, int mt, int tid = threadIdx.x) {
  const int i = tid & 15, g = (tid & 63) >> 4;
  return col_frag<NCOL>(lds, 8 * g, 8 * g + 4, state_row(mt, i & 3), state_row(mt, i >> 2) + (i & 3), tid);
}

// ---- T and P in operand order ----
//
// An A operand of row tile mt over the pair kp of token tiles: lane (i, g) row 16 mt + i, columns
// 32 kp + {4 g + 0..3, 16 + 4 g + 0..3}.  Only those that can hold a value are there: kp <= mt / 2 of a
// lower triangle, kp >= mt / 2 of a transpose.  Each is 64 lanes of 16 bytes (hi, then lo) or 32 (fp32).
template <typename E> struct Tri {
  static constexpr int C = Chunk<E>::C, NP = C / 32, kFrags = NP * (NP + 1);
  static constexpr int kFragBytes = 64 * 8 * sizeof(E);
  static constexpr int kHalfBytes = kFrags * kFragBytes;                    // one term
  static constexpr int kBytes = (sizeof(E) == 2 ? 2 : 1) * kHalfBytes;      // both
  // The place of (mt, kp), kp <= mt / 2; a transpose's (mt, kp) goes where the mirrored pair's is.
  static __device__ __forceinline__ int at(int mt, int kp) {
    const int p = mt >> 1;
    return p * (p + 1) + kp * 2 + (mt & 1);
  }
  static __device__ __forceinline__ int at_t(int mt, int kp) { return at(2 * (NP - 1 - (mt >> 1)) + (mt & 1), NP - 1 - kp); }
};
template <typename E> __device__ __forceinline__ typename Frag<E>::Raw tri_load(const char* base, int place) {  // base: in LDS
  using R = typename Frag<E>::Raw;
  return *reinterpret_cast<const R*>(base + place * Tri<E>::kFragBytes + (threadIdx.x & 63) * sizeof(R));
}
template <typename E> __device__ __forceinline__ Split<E> tri_load2(const char* base, int place) {
  Split<E> s;
  if constexpr (std::is_same_v<E, float>) {
    const f32x8 f = tri_load<float>(base, place);
    s.a = f.a;
    s.b = f.b;
  } else {
    s.hi = tri_load<bf16_t>(base, place);
    s.lo = tri_load<bf16_t>(base + Tri<bf16_t>::kHalfBytes, place);
  }
  return s;
}

// ---- the walks' workgroups ----
//
// WAVES waves hold 16 columns of a state each and do nothing but the chain of products; kLoaders more bring
// what a chunk needs from memory into LDS, three chunks ahead (two in registers, one in the other buffer), and
// carry the result columns away.  So the chain has no wait for memory in it and no registers go to loads.
// With few heads (WAVES = 2) each of these waves has a helper beside it, on a SIMD that would be idle, which
// takes over what is not part of the chain: of 160 matrix instructions a chunk 50.  They meet twice a chunk.

constexpr int kLoaders = 4, kLoadThreads = kLoaders * 64;

// A walk's LDS for one chunk.
template <typename E, int DKP, int WAVES> struct WalkTile {
  static constexpr int C = Chunk<E>::C;
  E K[C * Tile<E, DKP>::kRow];
  E Q[C * Tile<E, DKP>::kRow];
  char T[Tri<E>::kBytes];
  char P[Tri<E>::kBytes];
  float vec[3 * C];
  E V[C * 16 * WAVES];  // [token][column]: v, or the gradient of o
};
// The result columns of a chunk: bf16 as [column][token], fp32 as [token][column].
template <typename E, int WAVES> struct OutTile {
  static constexpr int C = Chunk<E>::C, kRow = sizeof(E) == 2 ? C + 4 : 16 * WAVES;
  E x[(sizeof(E) == 2 ? 16 * WAVES : C) * kRow];
};
// What a wave and its helper give each other.  Forward: the state and U as operands; backward: the tiles of
// P^T dO and of Q^T e^G dO.
template <typename E, int DKP, int WAVES> struct Exchange {
  static constexpr int C = Chunk<E>::C;
  static constexpr int kState = DKP * 16 * 4, kRows = C * 16 * 4;  // two bf16 terms or one fp32: four bytes a value
  char state[WAVES][kState];
  char rows[WAVES][kRows];
};
struct NoExchange {};
template <typename E> __device__ __forceinline__ void give(char* p, int n, const Split<E>& s) {
  reinterpret_cast<uint4*>(p)[2 * n * 64 + (threadIdx.x & 63)] = __builtin_bit_cast(uint4, first_half(s));
  reinterpret_cast<uint4*>(p)[(2 * n + 1) * 64 + (threadIdx.x & 63)] = __builtin_bit_cast(uint4, second_half(s));
}
template <typename E> __device__ __forceinline__ Split<E> take(const char* p, int n) {
  Split<E> s;
  const auto* q = reinterpret_cast<const decltype(first_half(s))*>(p);
  set_halves(s, q[2 * n * 64 + (threadIdx.x & 63)], q[(2 * n + 1) * 64 + (threadIdx.x & 63)]);
  return s;
}
__device__ __forceinline__ void give(char* p, int n, f32x4_t x) { reinterpret_cast<f32x4_t*>(p)[n * 64 + (threadIdx.x & 63)] = x; }
__device__ __forceinline__ f32x4_t take(const char* p, int n) { return reinterpret_cast<const f32x4_t*>(p)[n * 64 + (threadIdx.x & 63)]; }

// Two chunks where they fit the 160 KB, so that one is filled while the other is read.
template <typename E, int DKP, int WAVES>
constexpr int kWalkBuffers = 2 * (sizeof(WalkTile<E, DKP, WAVES>) + sizeof(OutTile<E, WAVES>)) <= 160 * 1024 ? 2 : 1;
constexpr int walk_waves(int waves) { return waves + (waves == 2 ? 2 : 0) + kLoaders; }  // of a workgroup

// A buffer resource over `bytes` bytes from p on (both the same for the wave): a load past them reads zero and
// a store past them does nothing, so short chunks and narrow heads need no branch.  A chunk's rows lie within
// 2^29 bytes; kNowhere, as a lane's offset, stays behind them for every row.
constexpr uint32_t kNowhere = 0x40000000u;
struct Buffer {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ Buffer(const void* p, int64_t bytes) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes > 0 ? bytes : 0));
    rs = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0, n, 0x00020000);
  }
  template <typename R> __device__ __forceinline__ R load(uint32_t off) const {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    const int o = static_cast<int>(off);
    if constexpr (sizeof(R) == 2) return __builtin_bit_cast(R, __builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0));
    else if constexpr (sizeof(R) == 4) return __builtin_bit_cast(R, __builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0));
    else return __builtin_bit_cast(R, static_cast<u32x4_t>(__builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0)));
  }
  __device__ __forceinline__ void store(uint32_t off, uint16_t x) const { __builtin_amdgcn_raw_buffer_store_b16(x, rs, static_cast<int>(off), 0, 0); }
  __device__ __forceinline__ void store(uint32_t off, float x) const {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), rs, static_cast<int>(off), 0, 0);
  }
  __device__ __forceinline__ void store16(uint32_t off, uint4 x) const {
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{x.x, x.y, x.z, x.w}, rs, static_cast<int>(off), 0, 0);
  }
};
// Bytes from the first element of `rows` rows of `cols` elements, ld apart, to the last one's end.
__device__ __forceinline__ int64_t rows_bytes(int rows, int64_t ld, int cols, int elem) {
  return rows > 0 ? ((rows - 1) * ld + cols) * elem : 0;
}

// The loaders' part: the next chunk's pieces in registers.
template <typename E, int DKP, int WAVES, bool WIDE, bool LEAN = false> struct Loader {  // LEAN: no queries, no scores
  using W = WalkTile<E, DKP, WAVES>;
  static constexpr int C = W::C, V = 16 / sizeof(E), kPieces = DKP / V, kStep = kLoadThreads / kPieces, kRows = C / kStep;
  static constexpr int kT = (Tri<E>::kBytes / 16 + kLoadThreads - 1) / kLoadThreads;
  static constexpr int kCols = 16 * WAVES, kVPieces = kCols / V, kVStep = kLoadThreads / kVPieces, kVRows = C / kVStep;
  static_assert(kLoadThreads % kPieces == 0 && C % kStep == 0 && 3 * C / 4 <= kLoadThreads && C % kVStep == 0);
  // as vectors: copies of uint4 alone, a structure, would leave the lean form's arrays in memory
  typedef uint32_t Vec __attribute__((ext_vector_type(4)));
  Vec k[kRows], q[LEAN ? 1 : kRows], t[kT], p[LEAN ? 1 : kT], vec, v[kVRows];
  int tid, row, col, vrow, vcol;  // of a thread's first pieces

  __device__ __forceinline__ Loader(int tid_)
      : tid(tid_), row(tid_ / kPieces), col(tid_ % kPieces * V), vrow(tid_ / kVPieces), vcol(tid_ % kVPieces * V) {}
  // Pieces past the end are some thread's twice: both write the same.
  __device__ __forceinline__ int piece(int n, int all) const { return min(tid + n * kLoadThreads, all - 1); }

  // cp: the first of the chunk's rows of v (or of the gradient of o), from this workgroup's column c0 on
  __device__ __forceinline__ void load(const Args& a, int chunk, int h, int64_t token, int len, const E* cp, int64_t ldc, int c0) {
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    const int hk = h / (a.H / a.Hk);
    const E *kp, *qp;
    int64_t lk, lq;
    int cols = DKP, krows = C;
    if (a.dense) {
      kp = static_cast<const E*>(a.k) + token * a.ldk + hk * a.dk;
      qp = static_cast<const E*>(a.q) + token * a.ldq + hk * a.dk;
      lk = a.ldk;
      lq = a.ldq;
      cols = a.dk;
      krows = len;
    } else {
      kp = static_cast<const E*>(a.kq) + (static_cast<int64_t>(chunk) * a.Hk + hk) * 2 * C * DKP;
      qp = kp + C * DKP;
      lk = lq = DKP;
    }
    const Buffer kb(kp, rows_bytes(krows, lk, cols, sizeof(E))), qb(qp, rows_bytes(krows, lq, cols, sizeof(E)));
    const uint32_t sk = static_cast<uint32_t>(lk * sizeof(E)), sq = static_cast<uint32_t>(lq * sizeof(E));
    const uint32_t at = col < cols ? col * sizeof(E) : kNowhere;
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      k[n] = kb.template load<Vec>(at + (row + n * kStep) * sk);
      if constexpr (!LEAN) q[n] = qb.template load<Vec>(at + (row + n * kStep) * sq);
    }
    const Vec* tp = reinterpret_cast<const Vec*>(a.t + item * Tri<E>::kBytes);
    const Vec* pp = reinterpret_cast<const Vec*>(a.p + item * Tri<E>::kBytes);
#pragma unroll
    for (int n = 0; n < kT; ++n) t[n] = tp[piece(n, Tri<E>::kBytes / 16)];
#pragma unroll
    for (int n = 0; n < (LEAN ? 0 : kT); ++n) p[n] = pp[piece(n, Tri<E>::kBytes / 16)];
    vec = reinterpret_cast<const Vec*>(a.vec + item * 3 * C)[piece(0, 3 * C / 4)];
    const int vcols = a.dv - c0;  // may be none
    const Buffer vb(cp, vcols > 0 ? rows_bytes(len, ldc, vcols, sizeof(E)) : 0);
    const uint32_t sv = static_cast<uint32_t>(ldc * sizeof(E));
    if constexpr (WIDE) {
      const uint32_t vat = vcol < vcols ? vcol * sizeof(E) : kNowhere;
#pragma unroll
      for (int n = 0; n < kVRows; ++n) v[n] = vb.template load<Vec>(vat + (vrow + n * kVStep) * sv);
    } else {
#pragma unroll
      for (int n = 0; n < kVRows; ++n) {
        E x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = vb.template load<E>(vcol + j < vcols ? (vcol + j) * sizeof(E) + (vrow + n * kVStep) * sv : kNowhere);
        __builtin_memcpy(&v[n], x, 16);
      }
    }
  }
  __device__ __forceinline__ void store(W& w) const {
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      const int at = Tile<E, DKP>::at(row + n * kStep, col);
      *reinterpret_cast<Vec*>(w.K + at) = k[n];
      if constexpr (!LEAN) *reinterpret_cast<Vec*>(w.Q + at) = q[n];
    }
#pragma unroll
    for (int n = 0; n < kT; ++n) reinterpret_cast<Vec*>(w.T)[piece(n, Tri<E>::kBytes / 16)] = t[n];
#pragma unroll
    for (int n = 0; n < (LEAN ? 0 : kT); ++n) reinterpret_cast<Vec*>(w.P)[piece(n, Tri<E>::kBytes / 16)] = p[n];
    reinterpret_cast<Vec*>(w.vec)[piece(0, 3 * C / 4)] = vec;
#pragma unroll
    for (int n = 0; n < kVRows; ++n) *reinterpret_cast<Vec*>(w.V + (vrow + n * kVStep) * kCols + vcol) = v[n];
  }
  // A chunk's result columns to memory (op: as cp).
  __device__ __forceinline__ void put(const Args& a, const OutTile<E, WAVES>& out, E* op, int64_t ldo, int len, int c0) const {
    const int cols = a.dv - c0;
    const Buffer ob(op, cols > 0 ? rows_bytes(len, ldo, cols, sizeof(E)) : 0);
    const uint32_t so = static_cast<uint32_t>(ldo * sizeof(E));
#pragma unroll
    for (int n = 0; n < kVRows; ++n) {
      int r, c;
      uint4 x;
      if constexpr (sizeof(E) == 2) {
        // 16 lanes: 16 tokens of eight columns
        typedef short v4s __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) const v4s lds_v4s;
        const int unit = tid / 16 + n * (kLoadThreads / 16), i = tid & 15;
        r = unit / kVPieces * 16;
        c = unit % kVPieces * 8;
        const auto p0 = (lds_v4s*)(out.x + (c + (i >> 2)) * out.kRow + r + 4 * (i & 3));
        const auto p1 = (lds_v4s*)(out.x + (c + 4 + (i >> 2)) * out.kRow + r + 4 * (i & 3));
        const v4s y[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p0),
                          __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p1)};
        x = __builtin_bit_cast(uint4, y);
        r += i;
      } else {
        r = vrow + n * kVStep;
        c = vcol;
        x = *reinterpret_cast<const uint4*>(out.x + r * out.kRow + c);
      }
      if constexpr (WIDE) {
        ob.store16(c < cols ? c * sizeof(E) + r * so : kNowhere, x);
      } else {
        E e[V];
        __builtin_memcpy(e, &x, 16);
#pragma unroll
        for (int j = 0; j < V; ++j) ob.store(c + j < cols ? (c + j) * sizeof(E) + r * so : kNowhere, e[j]);
      }
    }
  }
};

// The loaders' walk beside the others': from the first chunk on, BWD from the last back.  `in` and `out` are the
// head's first row of v (or of the gradient of o) and of the result; WIDE: both in 16-byte pieces; LEAN: there is no result.
template <typename E, int DKP, bool BWD, int WAVES, int BUF, bool MID, bool WIDE, bool LEAN = false, typename Tiles, typename Outs, typename S>
__device__ __forceinline__ void load_walk(const Args& a, const S& span, int h, int c0, Tiles& tiles, Outs& outs, const E* in, int64_t ld_in,
                                          E* out, int64_t ld_out) {
  constexpr int C = Chunk<E>::C;
  using L = Loader<E, DKP, WAVES, WIDE, LEAN>;
  const int tid = threadIdx.x - static_cast<int>(blockDim.x - kLoadThreads);
  // the chunks' pieces on their way, in turn; with one buffer, whose chunks are so wide, one of them fills the registers
  L even(tid), odd(tid);
  const int count = span.end - span.first;
  auto chunk_of = [&](int n) { return BWD ? span.end - 1 - min(n, count - 1) : span.first + min(n, count - 1); };
  auto load = [&](L& l, int n) {
    const int chunk = chunk_of(n);
    const int64_t token = span.token(chunk, C);
    l.load(a, chunk, h, token, span.len(chunk, C), in + token * ld_in + c0, ld_in, c0);
  };
  auto put = [&](int n) {
    if constexpr (!LEAN) {
      const int chunk = chunk_of(n);
      even.put(a, outs[n & (BUF - 1)], out + span.token(chunk, C) * ld_out + c0, ld_out, span.len(chunk, C), c0);
    }
  };
  auto step = [&](L& l, int n) {  // l has chunk n + 1
    if constexpr (BUF == 2) {
      l.store(tiles[(n + 1) & 1]);
      load(l, n + 3);
      if constexpr (MID) __syncthreads();
      if (n > 0) put(n - 1);
    } else {
      __syncthreads();  // the others are done with the chunk
      l.store(tiles[0]);
      load(l, n + 2);
      put(n);
    }
    __syncthreads();
  };
  if (count > 0) {
    load(even, 0);
    if constexpr (BUF == 2) load(odd, 1);
    even.store(tiles[0]);
    load(even, BUF);
  }
  __syncthreads();
  if constexpr (BUF == 2) {
    for (int n = 0; n < count; n += 2) {
      step(odd, n);
      if (n + 1 < count) step(even, n + 1);
    }
  } else {
    for (int n = 0; n < count; ++n) step(even, n);
  }
  if (BUF == 2 && count > 0) put(count - 1);
}

// What is written above stays above: the reads of a stage are under way while the one before is computed.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }
template <typename E> constexpr int kWhole = sizeof(E) == 2 ? 3 : 8;  // matrix instructions of a Whole operand and a tile
// N times a matrix instruction and then K others of the vector unit, which run while it does.
template <int N, int K> __device__ __forceinline__ void interleave() {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, K, 0);
  }
}

// c[n] += a[n] b over N tiles, the terms of b one after the other so that a tile's sums are far apart.
template <int N> __device__ __forceinline__ void mma_all(f32x4_t (&c)[N], const bf16x8_t (&a)[N], const Split<bf16_t>& b) {
#pragma unroll
  for (int n = 0; n < N; ++n) c[n] = mfma16(a[n], b.lo, c[n]);
#pragma unroll
  for (int n = 0; n < N; ++n) c[n] = mfma16(a[n], b.hi, c[n]);
}
template <int N> __device__ __forceinline__ void mma_all(f32x4_t (&c)[N], const bf16x8_t (&a)[N], const Whole<bf16_t>& b) {
#pragma unroll
  for (int n = 0; n < N; ++n) c[n] = mfma16(a[n], b.lo, c[n]);
#pragma unroll
  for (int n = 0; n < N; ++n) c[n] = mfma16(a[n], b.mid, c[n]);
#pragma unroll
  for (int n = 0; n < N; ++n) c[n] = mfma16(a[n], b.hi, c[n]);
}
// A walk's update of its state takes the state's tiles kGroup at a time: of 256 channels all at once, with the next
// operands on their way, would be twice the registers there are.
template <int ND> constexpr int kGroup = ND > 8 ? 8 : ND;
template <int N, int ND> __device__ __forceinline__ f32x4_t (&tiles_from(f32x4_t (&S)[ND], int t))[N] {
  return *reinterpret_cast<f32x4_t(*)[N]>(&S[t]);
}
// u += T x over the pair kp of token tiles; T lower triangular, TRANS its transpose.
template <typename E, bool TRANS = false, int NT>
__device__ __forceinline__ void tri_mul(f32x4_t (&u)[NT], const Split<E> (&t)[Tri<E>::kFrags], const Whole<E>& x, int kp) {
  using TR = Tri<E>;
  const int first = TRANS ? 0 : 2 * kp, end = TRANS ? 2 * kp + 2 : NT;
  if constexpr (std::is_same_v<E, float>) {
#pragma unroll
    for (int mt = first; mt < end; ++mt) u[mt] = mma(t[TRANS ? TR::at_t(mt, kp) : TR::at(mt, kp)], x, u[mt]);
  } else {
#pragma unroll
    for (int n = 0; n < 5; ++n)  // the smallest products first
#pragma unroll
      for (int mt = first; mt < end; ++mt) {
        const Split<E>& f = t[TRANS ? TR::at_t(mt, kp) : TR::at(mt, kp)];
        u[mt] = mfma16(n == 0 || n == 2 ? f.lo : f.hi, n == 1 ? x.lo : n == 0 || n == 3 ? x.mid : x.hi, u[mt]);
      }
  }
}
template <int N> __device__ __forceinline__ void mma_all(f32x4_t (&c)[N], const f32x8 (&a)[N], const Split<float>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int n = 0; n < N; ++n) c[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[n].a[j], b.a[j], c[n], 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int n = 0; n < N; ++n) c[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[n].b[j], b.b[j], c[n], 0, 0, 0);
}

// A walk's chunks: those of one sequence, and its tokens.
struct Span {
  int first, end;   // chunks
  int64_t token0, tokens;
  __device__ __forceinline__ int len(int chunk, int C) const {
    return static_cast<int>(min(static_cast<int64_t>(C), tokens - static_cast<int64_t>(chunk - first) * C));
  }
  __device__ __forceinline__ int64_t token(int chunk, int C) const { return token0 + static_cast<int64_t>(chunk - first) * C; }
};
template <int C> __device__ __forceinline__ Span span_of(const Args& a, int seq) {
  Span s;
  if (a.packed) {
    s.first = a.base[seq];
    s.end = a.base[seq + 1];
    s.token0 = s.tokens = 0;
    if (s.first < s.end) {
      const int4 head = a.table[s.first], tail = a.table[s.end - 1];
      s.token0 = head.x;
      s.tokens = tail.x + tail.y - head.x;
    }
  } else {  // seq: a piece of one
    const int n = seq % a.nseg * a.seg_chunks, whole = seq / a.nseg;
    s.first = whole * a.chunks_per_seq + n;
    s.end = whole * a.chunks_per_seq + min(n + a.seg_chunks, a.chunks_per_seq);
    s.token0 = static_cast<int64_t>(whole) * a.T + static_cast<int64_t>(n) * C;
    s.tokens = min(static_cast<int64_t>(a.T) - static_cast<int64_t>(n) * C, static_cast<int64_t>(a.seg_chunks) * C);
  }
  return s;
}

// Four rows r0 .. r0 + 3 of column col0 + i of a [..][LD] array, as a result tile has them.
template <int LD> __device__ __forceinline__ f32x4_t four_of(const bf16_t* lds, int r0, int col0) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const int i = threadIdx.x & 15;
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + (r0 + (i >> 2)) * LD + col0 + 4 * (i & 3)));
  f32x4_t f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = bf16_to_f32(static_cast<uint16_t>(x[j]));
  return f;
}
template <int LD> __device__ __forceinline__ f32x4_t four_of(const float* lds, int r0, int col0) {
  f32x4_t f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = lds[(r0 + j) * LD + col0 + (threadIdx.x & 15)];
  return f;
}
// A wave's 16 result columns of row tile mt.
template <int WAVES> __device__ __forceinline__ void out_tile(OutTile<bf16_t, WAVES>& o, int wave, int mt, f32x4_t x) {
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  *reinterpret_cast<uint2*>(o.x + (16 * wave + i) * o.kRow + 16 * mt + 4 * g) = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}
template <int WAVES> __device__ __forceinline__ void out_tile(OutTile<float, WAVES>& o, int wave, int mt, f32x4_t x) {
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) o.x[(16 * mt + 4 * g + r) * o.kRow + 16 * wave + i] = x[r];
}
// A wave's 16 columns of a [dk][dv] state to and from its result tiles.
template <int ND> __device__ __forceinline__ void state_load(const float* p, int dk, int dv, uint32_t at, f32x4_t (&S)[ND]) {
  const int g = (threadIdx.x & 63) >> 4;
  const Buffer b(p, p ? static_cast<int64_t>(dk) * dv * 4 : 0);
#pragma unroll
  for (int t = 0; t < ND; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[t][r] = b.load<float>(at + (state_row(t, g) + r) * dv * 4);
}
template <int ND> __device__ __forceinline__ void state_store(float* p, int dk, int dv, uint32_t at, const f32x4_t (&S)[ND]) {
  const int g = (threadIdx.x & 63) >> 4;
  const Buffer b(p, static_cast<int64_t>(dk) * dv * 4);
#pragma unroll
  for (int t = 0; t < ND; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) b.store(at + (state_row(t, g) + r) * dv * 4, S[t][r]);
}
template <typename E> __device__ __forceinline__ typename Frag<E>::Raw high(const Split<E>& s) {
  if constexpr (std::is_same_v<E, float>) return f32x8{s.a, s.b};
  else return s.hi;
}

// What the walks keep for the gradients (U, Y, the states before and the gradients of those after): fp32, or two terms of
// bf16, eight values' first and then their second.  In one term the gradients were up to 4e-3 off and not a rounding's
// 1.66e-3, and the gate's, in which large terms may cancel, up to 8e-2.
template <typename E> constexpr int kTerms = sizeof(E) == 2 ? 2 : 1;
template <typename E> constexpr uint32_t kKept = kTerms<E> * sizeof(E);  // bytes of a value
// `at`: bytes in front of the operand, all terms counted.
template <typename E> __device__ __forceinline__ void keep(const Buffer& b, uint32_t at, const Split<E>& s) {
  b.store16(at, __builtin_bit_cast(uint4, first_half(s)));
  b.store16(at + 16, __builtin_bit_cast(uint4, second_half(s)));
}

// ---- gates ----

// Log2 of the decay.  Below 2^-150 it is zero in fp32, and stays finite in the sums; a NaN stays one.
__device__ __forceinline__ float log2_decay(float z, int kind) {
  const float l = kind == TTT_GATE_LOG ? z : fminf(z, 0.0f) - log1pf(__expf(-fabsf(z)));
  const float l2 = z != z ? z : l * 1.4426950408889634f;
  return l2 < -150.0f ? -150.0f : l2;
}
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// One lane a token: the sum of log2 a up to it (in 64 bits: differences of far sums are exact enough for
// fp32), and eta; tokens that are not there keep the sum and have eta = 0.
template <typename E, int C>
__device__ __forceinline__ void gate_lane(const Args& a, const Where& w, int h, int t, double& G, float& eta, float& rest_sig, float& z) {
  z = 0.0f;
  eta = rest_sig = 0.0f;
  double l = 0.0;
  if (t < w.len) {
    const int64_t row = w.token + t;
    if (a.gate) {
      z = Elem<E>::ld(static_cast<const E*>(a.gate), row * a.ldg + h);
      l = log2_decay(z, a.gate_kind);
    }
    const float b = Elem<E>::ld(static_cast<const E*>(a.beta), row * a.ldb + h) + a.lr_bias;
    eta = a.lr_max / (1.0f + __expf(-b));
    rest_sig = 1.0f / (1.0f + __expf(b));
  }
#pragma unroll
  for (int d = 1; d < C; d <<= 1) {
    const double o = __shfl_up(l, d, 64);
    if ((threadIdx.x & 63) >= d) l += o;
  }
  G = l;
}

// Workgroups start in their order, so the longest sequences' walks are put first: 30011 tokens in 37 prompts, 20 heads,
// 284 us, in the prompts' own order 341.
__device__ __forceinline__ int walk_sequence(const Args& a, int chain) { return a.packed ? a.order[chain / a.H] : chain / a.H; }

// The waves of a walk's workgroup, and the workgroups that share a head's columns: four waves where that
// leaves a workgroup for every CU, else two with helpers.  30011 packed tokens of 20 heads of 128 bf16 (740 heads of
// sequences) take 284 us with four and 440 with two, 16 x 1024 tokens of 16 heads (256) 183 and 232, 4 x 4096 (64) 295 and
// 221.  Of 256 channels, four: helpers' part would not fit beside two chunks.
template <int DKP, typename F> hipError_t by_waves(const Args& a, F&& f) {
  const int64_t columns = a.dvp / 16;
  if constexpr (DKP == 256) return f(std::integral_constant<int, 4>{}, static_cast<int>((columns + 3) / 4));
  else if (static_cast<int64_t>(a.B) * a.nseg * a.H * ((columns + 3) / 4) >= 256) return f(std::integral_constant<int, 4>{}, static_cast<int>((columns + 3) / 4));
  else return f(std::integral_constant<int, 2>{}, static_cast<int>((columns + 1) / 2));
}

// Workgroups go to the eight XCDs in turn, each with an L2 of its own.  Those that share a head's keys and
// queries are put on one, the heads (chains) on all in turn: in long runs they are a sequence's.
inline uint32_t walk_grid(const Args& a, int groups) { return static_cast<uint32_t>((static_cast<int64_t>(a.B) * a.nseg * a.H + 7) / 8 * 8 * groups); }
__device__ __forceinline__ int walk_chain(int groups) { return static_cast<int>(blockIdx.x / 8 / groups * 8 + blockIdx.x % 8); }
__device__ __forceinline__ int walk_group(int groups) { return static_cast<int>(blockIdx.x / 8 % groups); }

// The chunks' T and P into the workspace (ttt_delta.hip; BWD: the transposes), and the backward's three
// kernels (ttt_delta_bwd.hip).
template <typename E, int DKP, bool BWD> hipError_t launch_prep(const Args& a, hipStream_t s);
template <typename E, int DKP> hipError_t launch_bwd(const Args& a, hipStream_t s);

}  // namespace delta
}  // namespace ttt
