// Gated delta rule: chunk table, chunk preparation, forward sweep and single-token step (see
// ttt_delta_common.h for the mathematics).

#include "ttt_delta_common.h"

namespace ttt {
namespace delta {
namespace {

constexpr int kPlanThreads = 1024;

// The chunk table of packed sequences: entries of seq_starts are held to 0 .. n and to ascend,
// so whatever they are, the chunks fit the table and the tokens the buffers.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int* starts, int B, int n, int C, int slots, int* edge, int* base,
                                                            int4* table, int* order) {
  __shared__ int part[kPlanThreads / 64], near_base[kPlanThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // running maximum of the starts
  int carry = 0;
  for (int i0 = 0; i0 <= B; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int m = i <= B ? min(max(starts[i], 0), n) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(m, d, 64);
      if (lane >= d) m = max(m, o);
    }
    if (lane == 63) part[wave] = m;
    __syncthreads();
    int before = carry, all = carry;
    for (int j = 0; j < kPlanThreads / 64; ++j) {
      if (j < wave) before = max(before, part[j]);
      all = max(all, part[j]);
    }
    if (i <= B) edge[i] = max(m, before);
    carry = all;
    __syncthreads();
  }
  // sums of the chunk counts
  carry = 0;
  for (int i0 = 0; i0 <= B; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int c = i < B ? (edge[i + 1] - edge[i] + C - 1) / C : 0;
    const int own = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(c, d, 64);
      if (lane >= d) c += o;
    }
    if (lane == 63) part[wave] = c;
    __syncthreads();
    int before = carry, all = carry;
    for (int j = 0; j < kPlanThreads / 64; ++j) {
      if (j < wave) before += part[j];
      all += part[j];
    }
    if (i <= B) base[i] = before + c - own;
    if (i < kPlanThreads) near_base[i] = before + c - own;  // for the search below
    carry = all;
    __syncthreads();
  }
  // the sequences by their chunks, the most first, of up to 1023.  More keep their own order: a long one at the end of
  // many short ones is then walked last, and by itself
  for (int i = threadIdx.x; i < B; i += kPlanThreads) {
    int rank = i;
    if (B < kPlanThreads) {
      const int own = near_base[i + 1] - near_base[i];
      rank = 0;
      for (int j = 0; j < B; ++j) {
        const int c = near_base[j + 1] - near_base[j];
        rank += c > own || (c == own && j < i);
      }
    }
    order[rank] = i;
  }
  const int total = carry;
  for (int c = threadIdx.x; c < slots; c += kPlanThreads) {
    int4 w = {0, -1, 0, 0};
    if (c < total) {
      int lo = 0, hi = B;  // the last sequence whose base is <= c
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((B < kPlanThreads ? near_base[mid] : base[mid]) <= c) lo = mid;
        else hi = mid;
      }
      const int first = edge[lo] + (c - base[lo]) * C;
      w = {first, min(C, edge[lo + 1] - first), lo, 0};
    }
    table[c] = w;
  }
}

// ---- T and P of every chunk ----

constexpr int kPrepThreads = 256;

// 16 x 16 blocks of a [C][C + 4] fp32 matrix as operands of v_mfma_f32_16x16x4_f32.
template <int LD> __device__ __forceinline__ f32x4_t block_row(const float* m, int bi, int bj) {
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  return *reinterpret_cast<const f32x4_t*>(m + (16 * bi + i) * LD + 16 * bj + 4 * g);
}
template <int LD> __device__ __forceinline__ f32x4_t block_col(const float* m, int bi, int bj) {
  const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  f32x4_t f;
#pragma unroll
  for (int r = 0; r < 4; ++r) f[r] = m[(16 * bi + 4 * g + r) * LD + 16 * bj + i];
  return f;
}

// A [C][C] fp32 matrix in operand order, hi and lo for bf16; TRANS: its transpose.
template <typename E, int LD, bool TRANS>
__device__ __forceinline__ void tri_store(const float* m, char* dst) {
  using T = Tri<E>;
  constexpr int kThreads = kPrepThreads;
  for (int idx = threadIdx.x; idx < T::kFrags * 64; idx += kThreads) {
    const int place = idx >> 6, lane = idx & 63, i = lane & 15, g = lane >> 4;
    const int p = place < 2 ? 0 : 1, kp = (place - p * (p + 1)) >> 1, mt = 2 * p + (place & 1);
    f32x4_t x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int row = 16 * mt + i, col = 32 * kp + 16 * h + 4 * g + j;
        if (TRANS) {  // the mirrored pair of the transpose
          row = 16 * (2 * (T::NP - 1 - p) + (mt & 1)) + i;
          col = 32 * (T::NP - 1 - kp) + 16 * h + 4 * g + j;
        }
        x[h][j] = TRANS ? m[col * LD + row] : m[row * LD + col];
      }
    if constexpr (std::is_same_v<E, float>) {
      *reinterpret_cast<f32x8*>(dst + place * T::kFragBytes + lane * 32) = f32x8{x[0], x[1]};
    } else {
      const Split<bf16_t> s(x[0], x[1]);
      *reinterpret_cast<bf16x8_t*>(dst + place * T::kFragBytes + lane * 16) = s.hi;
      *reinterpret_cast<bf16x8_t*>(dst + T::kHalfBytes + place * T::kFragBytes + lane * 16) = s.lo;
    }
  }
}

// T = (1 + A)^-1 by blocks of 16: the diagonal ones by forward substitution, a column a lane, then
// T_ij = -T_ii sum_{j<=l<i} A_il T_lj one diagonal after the other, all in fp32.
template <int C, int LD> __device__ __forceinline__ void invert(const float* A, float* T) {
  constexpr int NB = C / 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  if (wave < NB && lane < 16) {
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int l = 0; l < r; ++l) s -= A[(16 * wave + r) * LD + 16 * wave + l] * x[l];
      x[r] = s;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) T[(16 * wave + r) * LD + 16 * wave + lane] = x[r];
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < NB; ++d) {
    if (wave < NB - d) {
      const int bj = wave, bi = wave + d;
      f32x4_t s = zero4();
#pragma unroll
      for (int l = 0; l < d; ++l) s = mfma16(block_row<LD>(A, bi, bj + l), block_col<LD>(T, bj + l, bj), s);
      f32x4_t x = zero4();
      x = mfma16(block_row<LD>(T, bi, bi), s, x);
#pragma unroll
      for (int r = 0; r < 4; ++r) T[(16 * bi + 4 * g + r) * LD + 16 * bj + i] = -x[r];
    }
    __syncthreads();
  }
}

// A chunk and head a workgroup: its gates' sums, K K^T and Q K^T (row tile w by wave w), the inverse.
// BWD writes the transposes.  Both in two terms: with the scores in one, O was 2.2e-3 off and not a rounding's 1.66e-3
// (a forward over 30011 packed tokens of 20 heads takes 5 % longer so).  It is bound by the latency of its stages, so LDS is
// used over and over: 36 KB let four workgroups share a CU.  4096 chunks and heads of 128 bf16 60 us (93 with 53 KB,
// three workgroups and the loads behind the gates' sums).
template <typename E, int DKP, bool BWD>
__global__ __launch_bounds__(kPrepThreads) void prep_kernel(Args a) {
  constexpr int C = Chunk<E>::C, NT = C / 16, LD = C + 4, V = 16 / sizeof(E), kPieces = DKP / V, kRows = C * kPieces / kPrepThreads;
  using Lds = Tile<E, DKP>;
  // A and T take the place of the keys and queries, the scores that of A
  constexpr size_t kRowsBytes = 2 * C * Lds::kRow * sizeof(E), kSquares = 2 * C * LD * sizeof(float);
  __shared__ __attribute__((aligned(16))) char pool[kRowsBytes > kSquares ? kRowsBytes : kSquares];
  E* K = reinterpret_cast<E*>(pool);
  E* Q = K + C * Lds::kRow;
  float* A = reinterpret_cast<float*>(pool);
  float* T = A + C * LD;
  __shared__ double G[C];
  __shared__ float eta[C];
  const int chunk = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const Where w = locate<C>(a, chunk);
  if (w.len < 0) return;
  const int hk = h / (a.H / a.Hk);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
  const E* kp = static_cast<const E*>(a.k) + w.token * a.ldk + hk * a.dk;
  const E* qp = static_cast<const E*>(a.q) + w.token * a.ldq + hk * a.dk;
  uint4 kr[kRows], qr[kRows];
  if (a.dense) {  // on their way while the gates are summed
    const Buffer kb(kp, rows_bytes(w.len, a.ldk, a.dk, sizeof(E))), qb(qp, rows_bytes(w.len, a.ldq, a.dk, sizeof(E)));
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      const int x = threadIdx.x + n * kPrepThreads, row = x / kPieces, col = x % kPieces * V;
      kr[n] = kb.template load<uint4>(col < a.dk ? (row * static_cast<uint32_t>(a.ldk) + col) * sizeof(E) : kNowhere);
      qr[n] = qb.template load<uint4>(col < a.dk ? (row * static_cast<uint32_t>(a.ldq) + col) * sizeof(E) : kNowhere);
    }
  }
  if (wave == 0) {
    double Gt;
    float et, rs, z;
    gate_lane<E, C>(a, w, h, lane, Gt, et, rs, z);
    const double last = __shfl(Gt, C - 1, 64);
    if (lane < C) {
      G[lane] = Gt;
      eta[lane] = et;
      float* vec = a.vec + item * 3 * C + lane;
      vec[0] = exp2_(static_cast<float>(Gt));
      vec[C] = exp2_(static_cast<float>(last - Gt));
      vec[2 * C] = et;
    }
  }
  if (a.dense) {
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      const int x = threadIdx.x + n * kPrepThreads, at = Lds::at(x / kPieces, x % kPieces * V);
      *reinterpret_cast<uint4*>(K + at) = kr[n];
      *reinterpret_cast<uint4*>(Q + at) = qr[n];
    }
  } else {
    stage<E, C, DKP, kPrepThreads>(K, kp, a.ldk, w.len, a.dk, a.wide_k);
    stage<E, C, DKP, kPrepThreads>(Q, qp, a.ldq, w.len, a.dk, a.wide_q);
  }
  __syncthreads();
  if (!a.dense && h % (a.H / a.Hk) == 0) {  // the walks' copy
    E* dst = static_cast<E*>(a.kq) + (static_cast<int64_t>(chunk) * a.Hk + hk) * 2 * C * DKP;
    for (int x = threadIdx.x; x < 2 * C * kPieces; x += kPrepThreads) {
      const int row = x / kPieces, col = (x % kPieces) * V;
      const E* src = row < C ? K + Lds::at(row, col) : Q + Lds::at(row - C, col);
      *reinterpret_cast<uint4*>(dst + row * DKP + col) = *reinterpret_cast<const uint4*>(src);
    }
  }
  const int mt = wave;  // row tile; NT waves have one
  f32x4_t kk[NT], qk[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) kk[nt] = qk[nt] = zero4();
  if (mt < NT) {
    // all column tiles, those above the diagonal too: no branch between the products
#pragma unroll
    for (int p = 0; p < DKP / 32; ++p) {
      typename Frag<E>::Raw b[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) b[nt] = row_frag<DKP>(K, 16 * nt + i, 32 * p + 8 * g);
      const auto ka = row_frag<DKP>(K, 16 * mt + i, 32 * p + 8 * g), qa = row_frag<DKP>(Q, 16 * mt + i, 32 * p + 8 * g);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        kk[nt] = mma(ka, b[nt], kk[nt]);
        qk[nt] = mma(qa, b[nt], qk[nt]);
      }
    }
  }
  __syncthreads();
  if (mt < NT) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * mt + 4 * g + r, col = 16 * nt + i;
        const float d = row >= col ? exp2_(static_cast<float>(G[row] - G[col])) : 0.0f;
        A[row * LD + col] = row > col ? eta[row] * d * kk[nt][r] : 0.0f;
        T[row * LD + col] = 0.0f;
        qk[nt][r] = row >= col ? a.scale * d * qk[nt][r] : 0.0f;
      }
  }
  __syncthreads();
  invert<C, LD>(A, T);
  tri_store<E, LD, BWD>(T, a.t + item * Tri<E>::kBytes);
  if (mt < NT) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r) A[(16 * mt + 4 * g + r) * LD + 16 * nt + i] = qk[nt][r];
  }
  __syncthreads();
  tri_store<E, LD, BWD>(A, a.p + item * Tri<E>::kBytes);
}

// ---- forward walk ----

// The state that enters a sequence or a piece of one (NULL: zero), and where the one that leaves it goes.
__device__ __forceinline__ const float* entering(const Args& a, int seq, int h) {
  const int64_t at = (static_cast<int64_t>(seq) * a.H + h) * a.dk * a.dv;
  return a.nseg > 1 ? a.seg_states + at : a.s0 ? a.s0 + at : nullptr;
}
__device__ __forceinline__ float* leaving(const Args& a, int seq, int h) {
  if (!a.s_final || seq % a.nseg != a.nseg - 1) return nullptr;
  return a.s_final + (static_cast<int64_t>(seq / a.nseg) * a.H + h) * a.dk * a.dv;
}

// The chain (waves 0 .. WAVES - 1) and its helpers (the next WAVES) where there are few heads.  First half of a
// chunk: K S, U and, by the helper, Q S; second half: the next state and, by the helper, O += P U.  A chunk of 64 x 128
// bf16 takes 2.3 us (3.4 where every CU has one and keeps what a backward needs), which is the chain's own: 110 matrix
// instructions and about 450 vector instructions, one in 5.5 cycles from one wave.  64 chunks of 64 heads with what a
// backward needs 221 us, with four chain waves a workgroup instead 295.
template <typename E, int DKP, int WAVES, bool KEEP, typename Tiles, typename Outs>
__device__ __forceinline__ void help_fwd_or_chain(const Args& a, const Span& span, int seq, int h, int grp, Tiles& tiles, Outs& outs,
                                                  Exchange<E, DKP, WAVES>& exchange) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, ND = DKP / 16, NK = DKP / 32;
  using TR = Tri<E>;
  using Raw = typename Frag<E>::Raw;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const bool helper = threadIdx.x >= WAVES * 64;
  const int wave = (threadIdx.x >> 6) % WAVES, col = (grp * WAVES + wave) * 16 + i;
  char* states = exchange.state[wave];
  char* us = exchange.rows[wave];
  if (helper) {
    const bool live = col < a.dvp;
    const uint32_t u_at = live ? (col * C + 8 * g) * kKept<E> : kNowhere, b_at = live ? (col * DKP + 8 * g) * kKept<E> : kNowhere;
    __syncthreads();
    for (int chunk = span.first; chunk < span.end; ++chunk) {
      const auto& w = tiles[(chunk - span.first) & 1];
      const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
      const Buffer kept(KEEP ? static_cast<char*>(a.before) + item * a.dvp * DKP * kKept<E> : nullptr, static_cast<int64_t>(a.dvp) * DKP * kKept<E>);
      f32x4_t o[NT];
      Raw rows[2][NT];
      Split<E> s[2];
      auto read = [&](int kp) {
        s[kp & 1] = take<E>(states, kp);
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) rows[kp & 1][mt] = row_frag<DKP>(w.Q, 16 * mt + i, 32 * kp + 8 * g);
      };
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) o[mt] = zero4();
      read(0);
#pragma unroll
      for (int kp = 0; kp < NK; ++kp) {
        if (kp + 1 < NK) read(kp + 1);
        in_order();
        if constexpr (KEEP) keep<E>(kept, b_at + 32 * kp * kKept<E>, s[kp & 1]);
        mma_all(o, rows[kp & 1], s[kp & 1]);
        in_order();
      }
      Split<E> scores[TR::kFrags];
#pragma unroll
      for (int f = 0; f < TR::kFrags; ++f) scores[f] = tri_load2<E>(w.P, f);
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) o[mt] *= *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g) * a.scale;
      __syncthreads();
      const Buffer ub(KEEP ? static_cast<char*>(a.u) + item * a.dvp * C * kKept<E> : nullptr, static_cast<int64_t>(a.dvp) * C * kKept<E>);
#pragma unroll
      for (int kp = 0; kp < NP; ++kp) {
        const Split<E> u = take<E>(us, kp);
        if constexpr (KEEP) keep<E>(ub, u_at + 32 * kp * kKept<E>, u);
#pragma unroll
        for (int mt = 2 * kp; mt < NT; ++mt) o[mt] = mma(scores[TR::at(mt, kp)], u, o[mt]);
      }
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) out_tile(outs[(chunk - span.first) & 1], wave, mt, o[mt]);
      __syncthreads();
    }
    return;
  }
  const uint32_t s_at = col < a.dv ? col * 4 : kNowhere;
  f32x4_t S[ND];
  state_load(entering(a, seq, h), a.dk, a.dv, s_at, S);
  Split<E> s[NK];
#pragma unroll
  for (int kp = 0; kp < NK; ++kp) {
    s[kp] = Split<E>(S[2 * kp], S[2 * kp + 1]);
    give(states, kp, s[kp]);
  }
  __syncthreads();
  for (int chunk = span.first; chunk < span.end; ++chunk) {
    const auto& w = tiles[(chunk - span.first) & 1];
    f32x4_t ks[NT], gm[NT], et[NT], vt[NT], rest[NT];
    Raw rows[2][NT];
    auto read_rows = [&](int kp) {
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) rows[kp & 1][mt] = row_frag<DKP>(w.K, 16 * mt + i, 32 * kp + 8 * g);
    };
    Split<E> tri[TR::kFrags];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) ks[mt] = zero4();
    read_rows(0);
#pragma unroll
    for (int kp = 0; kp < NK; ++kp) {
      if (kp + 1 < NK) {
        read_rows(kp + 1);
      }
      if (kp + 2 == NK || NK == 1) {
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
          gm[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g);
          et[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 2 * C + 16 * mt + 4 * g);
          vt[mt] = four_of<16 * WAVES>(w.V, 16 * mt + 4 * g, 16 * wave);
        }
      }
      if (kp + 1 == NK) {
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) tri[f] = tri_load2<E>(w.T, f);
      }
      in_order();
      mma_all(ks, rows[kp & 1], s[kp]);
      in_order();
    }
    const float decay = w.vec[C - 1];
    Raw cols[2][ND];
    auto read_cols = [&](int kp) {
#pragma unroll
      for (int t = 0; t < ND; ++t) cols[kp & 1][t] = state_col<DKP>(w.K, 32 * kp, t);
    };
    f32x4_t u[NT];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      rest[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + C + 16 * mt + 4 * g);
      ks[mt] = et[mt] * (vt[mt] - gm[mt] * ks[mt]);
      u[mt] = zero4();
    }
    read_cols(0);
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Whole<E> rhs(ks[2 * kp], ks[2 * kp + 1]);
      tri_mul<E>(u, tri, rhs, kp);
    }
#pragma unroll
    for (int t = 0; t < ND; ++t) S[t] *= decay;
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) give(us, kp, Split<E>(u[2 * kp], u[2 * kp + 1]));
    __syncthreads();
    Whole<E> x(u[0] * rest[0], u[1] * rest[1]);
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      if (kp + 1 < NP) read_cols(kp + 1);
      in_order();
      mma_all(S, cols[kp & 1], x);
      if (kp + 1 < NP) {
        x = Whole<E>(u[2 * kp + 2] * rest[2 * kp + 2], u[2 * kp + 3] * rest[2 * kp + 3]);
        interleave<kWhole<E> * ND, 2>();
      }
      in_order();
    }
#pragma unroll
    for (int kp = 0; kp < NK; ++kp) {
      s[kp] = Split<E>(S[2 * kp], S[2 * kp + 1]);
      give(states, kp, s[kp]);
    }
    __syncthreads();
  }
  if (float* to = leaving(a, seq, h)) state_store(to, a.dk, a.dv, s_at, S);
}

// A wave holds 16 columns of a head's state in its result registers and walks the chunks.  The state and what
// is added to it are products of operands of two and three terms: its error does not grow with the length.  KEEP: what a
// backward needs is written.  30011 packed tokens of 20 heads of 128 bf16 284 us (323 under the profiler), 3.8 us a chunk of a workgroup: four
// chains share LDS, and the loads of 256 workgroups the memory.
template <typename E, int DKP, int WAVES, bool KEEP>
__global__ __launch_bounds__(walk_waves(WAVES) * 64, 1) void fwd_kernel(Args a, int groups) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, ND = DKP / 16, NK = DKP / 32, kBuf = kWalkBuffers<E, DKP, WAVES>;
  constexpr int kMma = sizeof(E) == 2 ? 1 : 4;  // matrix instructions of an operand's term
  constexpr int TG = kGroup<ND>, NG = ND / TG;
  using TR = Tri<E>;
  using Raw = typename Frag<E>::Raw;
  __shared__ __attribute__((aligned(16))) WalkTile<E, DKP, WAVES> tiles[kBuf];
  __shared__ __attribute__((aligned(16))) OutTile<E, WAVES> outs[kBuf];
  __shared__ __attribute__((aligned(16))) std::conditional_t<WAVES == 2, Exchange<E, DKP, WAVES>, NoExchange> exchange;
  const int grp = walk_group(groups), chain = walk_chain(groups);
  if (chain >= a.B * a.nseg * a.H) return;
  const int h = chain % a.H, seq = walk_sequence(a, chain);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const Span span = span_of<C>(a, seq);
  constexpr bool HELP = WAVES == 2;
  if (wave >= WAVES + (HELP ? WAVES : 0)) {
    const E* in = static_cast<const E*>(a.v) + static_cast<int64_t>(h) * a.dv;
    E* out = static_cast<E*>(a.o) + static_cast<int64_t>(h) * a.dv;
    const int64_t ldo = static_cast<int64_t>(a.H) * a.dv;
    if (a.wide_v && a.wide_o) load_walk<E, DKP, false, WAVES, kBuf, HELP, true>(a, span, h, grp * WAVES * 16, tiles, outs, in, a.ldv, out, ldo);
    else load_walk<E, DKP, false, WAVES, kBuf, HELP, false>(a, span, h, grp * WAVES * 16, tiles, outs, in, a.ldv, out, ldo);
    return;
  }
  if constexpr (HELP) {
    help_fwd_or_chain<E, DKP, WAVES, KEEP>(a, span, seq, h, grp, tiles, outs, exchange);
    return;
  }
  const int col = (grp * WAVES + wave) * 16 + i;
  const bool live = col < a.dvp;
  const uint32_t s_at = col < a.dv ? col * 4 : kNowhere;
  f32x4_t S[ND];
  state_load(entering(a, seq, h), a.dk, a.dv, s_at, S);
  __builtin_amdgcn_s_waitcnt(0);  // here, so that the loop has no wait for memory
  const uint32_t u_at = live ? (col * C + 8 * g) * kKept<E> : kNowhere, b_at = live ? (col * DKP + 8 * g) * kKept<E> : kNowhere;
  __syncthreads();
  for (int chunk = span.first; chunk < span.end; ++chunk) {
    const WalkTile<E, DKP, WAVES>& w = tiles[(chunk - span.first) & (kBuf - 1)];
    OutTile<E, WAVES>& out = outs[(chunk - span.first) & (kBuf - 1)];
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    // K S and Q S: rows of the next 32 channels are read, and their part of the state split, while these are multiplied
    f32x4_t ko[2 * NT];
    Raw rows[2][2 * NT];
    auto read_rows = [&](int kp) {
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) {
        rows[kp & 1][mt] = row_frag<DKP>(w.K, 16 * mt + i, 32 * kp + 8 * g);
        rows[kp & 1][NT + mt] = row_frag<DKP>(w.Q, 16 * mt + i, 32 * kp + 8 * g);
      }
    };
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) ko[n] = zero4();
    read_rows(0);
    Split<E> tri[TR::kFrags];
    f32x4_t gm[NT], et[NT], rest[NT], vt[NT];
    const Buffer kept(KEEP ? static_cast<char*>(a.before) + item * a.dvp * DKP * kKept<E> : nullptr, static_cast<int64_t>(a.dvp) * DKP * kKept<E>);
    Split<E> s(S[0], S[1]);
#pragma unroll
    for (int kp = 0; kp < NK; ++kp) {
      if (kp + 1 < NK) {
        read_rows(kp + 1);
      } else {
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
          gm[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g);
          et[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 2 * C + 16 * mt + 4 * g);
          vt[mt] = four_of<16 * WAVES>(w.V, 16 * mt + 4 * g, 16 * wave);
        }
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) tri[f] = tri_load2<E>(w.T, f);
      }
      if constexpr (KEEP) keep<E>(kept, b_at + 32 * kp * kKept<E>, s);
      in_order();
      mma_all(ko, rows[kp & 1], s);
      if (kp + 1 < NK) {
        s = Split<E>(S[2 * kp + 2], S[2 * kp + 3]);
        interleave<4 * NT * kMma, 2>();
      }
      in_order();
    }
    // eta (V - e^G K S), U = T (that)
    const float decay = w.vec[C - 1];
    Raw cols[2][TG];
    auto read_cols = [&](int n) {  // the pairs of token tiles, each by groups of the state's tiles
#pragma unroll
      for (int t = 0; t < TG; ++t) cols[n & 1][t] = state_col<DKP>(w.K, 32 * (n / NG), n % NG * TG + t);
    };
    read_cols(0);
    f32x4_t o[NT], u[NT];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      rest[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + C + 16 * mt + 4 * g);
      ko[mt] = et[mt] * (vt[mt] - gm[mt] * ko[mt]);
      u[mt] = zero4();
    }
    in_order();
    // the products with T leave room for what the next stages need
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Whole<E> rhs(ko[2 * kp], ko[2 * kp + 1]);
      tri_mul<E>(u, tri, rhs, kp);
    }
#pragma unroll
    for (int t = 0; t < ND; ++t) S[t] *= decay;
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) o[mt] = ko[NT + mt] * (a.scale * gm[mt]);
    in_order();
    // S = e^{G_C} S + K^T (e^{G_C - G} U);  O += P U
    Split<E> scores[TR::kFrags];
    const Buffer ub(KEEP ? static_cast<char*>(a.u) + item * a.dvp * C * kKept<E> : nullptr, static_cast<int64_t>(a.dvp) * C * kKept<E>);
    Split<E> us[NP];
    Whole<E> x(u[0] * rest[0], u[1] * rest[1]);
#pragma unroll
    for (int n = 0; n < NP * NG; ++n) {
      const int kp = n / NG;
      if (n + 1 < NP * NG) {
        read_cols(n + 1);
      } else {
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) scores[f] = tri_load2<E>(w.P, f);
      }
      in_order();
      mma_all(tiles_from<TG>(S, n % NG * TG), cols[n & 1], x);
      if (n % NG == 0) us[kp] = Split<E>(u[2 * kp], u[2 * kp + 1]);
      if (n % NG == NG - 1 && kp + 1 < NP) x = Whole<E>(u[2 * kp + 2] * rest[2 * kp + 2], u[2 * kp + 3] * rest[2 * kp + 3]);
      interleave<kWhole<E> * TG, 3>();
      in_order();
    }
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      if constexpr (KEEP) keep<E>(ub, u_at + 32 * kp * kKept<E>, us[kp]);
#pragma unroll
      for (int mt = 2 * kp; mt < NT; ++mt) o[mt] = mma(scores[TR::at(mt, kp)], us[kp], o[mt]);
    }
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) out_tile(out, wave, mt, o[mt]);
    if constexpr (kBuf == 1) __syncthreads();
    __syncthreads();
  }
  if (float* to = leaving(a, seq, h)) state_store(to, a.dk, a.dv, s_at, S);
}

// ---- pieces of a long sequence ----
//
// Over some chunks the state maps to M S + N: M is where they take the columns of the identity without any
// values, N where they take a zero state.  So where there are few heads the pieces of a sequence are walked at
// the same time twice, first for their maps (dk + dv columns, no outputs), then from the states that the maps give.

constexpr int kMapWaves = 4;

// The maps: [piece][H][dkp][dvp + dkp], N before M.  The last piece's is not needed.  Seven of eight pieces of 131072
// tokens, 16 heads of 128 bf16, 1061 us; the whole walk after it 763, in one piece 4822.
template <typename E, int DKP>
__global__ __launch_bounds__((kMapWaves + kLoaders) * 64, 1) void map_kernel(Args a, int groups, float* maps) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, ND = DKP / 16, NK = DKP / 32, WAVES = kMapWaves;
  constexpr int kBuf = kWalkBuffers<E, DKP, WAVES>;
  using TR = Tri<E>;
  using Raw = typename Frag<E>::Raw;
  __shared__ __attribute__((aligned(16))) WalkTile<E, DKP, WAVES> tiles[kBuf];
  const int grp = walk_group(groups), chain = walk_chain(groups);
  if (chain >= a.B * a.nseg * a.H) return;
  const int h = chain % a.H, seq = walk_sequence(a, chain);
  if (seq % a.nseg == a.nseg - 1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const Span span = span_of<C>(a, seq);
  if (wave >= WAVES) {
    const E* in = static_cast<const E*>(a.v) + static_cast<int64_t>(h) * a.dv;
    if (a.wide_v) load_walk<E, DKP, false, WAVES, kBuf, false, true, true>(a, span, h, grp * WAVES * 16, tiles, tiles, in, a.ldv, static_cast<E*>(nullptr), 0);
    else load_walk<E, DKP, false, WAVES, kBuf, false, false, true>(a, span, h, grp * WAVES * 16, tiles, tiles, in, a.ldv, static_cast<E*>(nullptr), 0);
    return;
  }
  const int col = (grp * WAVES + wave) * 16 + i, width = a.dvp + DKP;
  f32x4_t S[ND];
#pragma unroll
  for (int t = 0; t < ND; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[t][r] = state_row(t, g) + r == col - a.dvp ? 1.0f : 0.0f;
  __syncthreads();
  for (int chunk = span.first; chunk < span.end; ++chunk) {
    const auto& w = tiles[(chunk - span.first) & (kBuf - 1)];
    f32x4_t ks[NT], u[NT], gm[NT], et[NT], vt[NT], rest[NT];
    Raw rows[2][NT];
    auto read_rows = [&](int kp) {
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) rows[kp & 1][mt] = row_frag<DKP>(w.K, 16 * mt + i, 32 * kp + 8 * g);
    };
    Split<E> tri[TR::kFrags];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) ks[mt] = u[mt] = zero4();
    read_rows(0);
    Split<E> s(S[0], S[1]);
#pragma unroll
    for (int kp = 0; kp < NK; ++kp) {
      if (kp + 1 < NK) {
        read_rows(kp + 1);
      } else {
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
          gm[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g);
          et[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 2 * C + 16 * mt + 4 * g);
          vt[mt] = four_of<16 * WAVES>(w.V, 16 * mt + 4 * g, 16 * wave);
        }
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) tri[f] = tri_load2<E>(w.T, f);
      }
      in_order();
      mma_all(ks, rows[kp & 1], s);
      if (kp + 1 < NK) s = Split<E>(S[2 * kp + 2], S[2 * kp + 3]);
      in_order();
    }
    const float decay = w.vec[C - 1];
    Raw cols[ND];
    auto read_cols = [&](int kp) {
#pragma unroll
      for (int t = 0; t < ND; ++t) cols[t] = state_col<DKP>(w.K, 32 * kp, t);
    };
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      rest[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + C + 16 * mt + 4 * g);
      ks[mt] = et[mt] * (vt[mt] - gm[mt] * ks[mt]);
    }
    read_cols(0);
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) tri_mul<E>(u, tri, Whole<E>(ks[2 * kp], ks[2 * kp + 1]), kp);
#pragma unroll
    for (int t = 0; t < ND; ++t) S[t] *= decay;
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Whole<E> x(u[2 * kp] * rest[2 * kp], u[2 * kp + 1] * rest[2 * kp + 1]);
      mma_all(S, cols, x);
      if (kp + 1 < NP) read_cols(kp + 1);
    }
    if constexpr (kBuf == 1) __syncthreads();
    __syncthreads();
  }
  if (col < width) {
    float* to = maps + (static_cast<int64_t>(seq) * a.H + h) * DKP * width + col;
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) to[static_cast<int64_t>(state_row(t, g) + r) * width] = S[t][r];
  }
}

// The states that enter the pieces, one after the other: 16 columns of a head a workgroup, 16 rows a wave.
template <typename E, int DKP>
__global__ __launch_bounds__(DKP * 4) void join_kernel(Args a, const float* maps, float* states) {
  constexpr int NK = DKP / 32;
  __shared__ f32x4_t S[DKP / 16][64];
  const int groups = a.dvp / 16, grp = blockIdx.x % groups, h = blockIdx.x / groups % a.H, seq = blockIdx.x / groups / a.H;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int col = 16 * grp + i, width = a.dvp + DKP;
  f32x4_t x;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 16 * wave + 4 * g + r;
    x[r] = a.s0 && row < a.dk && col < a.dv ? a.s0[((static_cast<int64_t>(seq) * a.H + h) * a.dk + row) * a.dv + col] : 0.0f;
  }
  for (int n = 0; n < a.nseg; ++n) {
    const int64_t piece = (static_cast<int64_t>(seq) * a.nseg + n) * a.H + h;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * wave + 4 * g + r;
      if (row < a.dk && col < a.dv) states[(piece * a.dk + row) * a.dv + col] = x[r];
    }
    if (n + 1 == a.nseg) return;
    S[wave][lane] = x;
    const float* m = maps + piece * DKP * width;
    f32x4_t c, row[2 * NK];
#pragma unroll
    for (int kp = 0; kp < 2 * NK; ++kp)
      row[kp] = *reinterpret_cast<const f32x4_t*>(m + static_cast<int64_t>(16 * wave + i) * width + a.dvp + 16 * kp + 4 * g);
#pragma unroll
    for (int r = 0; r < 4; ++r) c[r] = m[static_cast<int64_t>(16 * wave + 4 * g + r) * width + col];
    __syncthreads();
#pragma unroll
    for (int kp = 0; kp < 2 * NK; ++kp) c = mfma16(row[kp], S[kp][lane], c);
    __syncthreads();
    x = c;
  }
}

// ---- one token ----

constexpr int kStepThreads = 256;

// A workgroup has kStepCols columns of one head's state of one row, a thread a run of the dk rows of one
// column; the three sums over dk meet in LDS.  256 rows of 16 heads of 128 x 128 (537 MB) 114 us, 4.7 TB/s; 8 rows
// 7.1 us, the latency of slot, state and sums.  Rows that name one slot are consecutive tokens of it, in
// row order: the first of them does them all.
constexpr int kStepCols = 32, kStepRuns = kStepThreads / kStepCols;

struct StepArgs {
  int B, H, Hk, dk, dv, gate_kind, n_states, ncb;
  float scale, lr_max, lr_bias;
  int64_t ldq, ldk, ldv, ldg, ldb;
  const void* q;
  const void* k;
  const void* v;
  const void* gate;
  const void* beta;
  const int32_t* slots;
  const float* s;
  float* s_new;
  void* o;
};

template <typename E, int NR>  // NR: rows of the state a thread holds
__global__ __launch_bounds__(kStepThreads) void step_kernel(StepArgs a) {
  __shared__ float part[2][kStepRuns][kStepCols], kq_part[kStepRuns];
  __shared__ float ks[kStepRuns * NR], qs[kStepRuns * NR];
  __shared__ uint64_t same[kStepThreads / 64];
  static_assert(kStepRuns * NR <= kStepThreads);
  const int cb = blockIdx.x % a.ncb, h = blockIdx.x / a.ncb % a.H, b = blockIdx.x / a.ncb / a.H;
  const int hk = h / (a.H / a.Hk);
  const int c = threadIdx.x % kStepCols, run = threadIdx.x / kStepCols, col = cb * kStepCols + c;
  // a token's values; the first one's are on their way while its slot is looked for
  float kx, qx, vt, z, bt;
  auto fetch = [&](int64_t row) {
    const int x = threadIdx.x;
    kx = x < a.dk ? Elem<E>::ld(static_cast<const E*>(a.k), row * a.ldk + hk * a.dk + x) : 0.0f;
    qx = x < a.dk ? Elem<E>::ld(static_cast<const E*>(a.q), row * a.ldq + hk * a.dk + x) : 0.0f;
    vt = col < a.dv ? Elem<E>::ld(static_cast<const E*>(a.v), row * a.ldv + static_cast<int64_t>(h) * a.dv + col) : 0.0f;
    z = a.gate ? Elem<E>::ld(static_cast<const E*>(a.gate), row * a.ldg + h) : 0.0f;
    bt = Elem<E>::ld(static_cast<const E*>(a.beta), row * a.ldb + h);
  };
  fetch(b);
  int slot = b;
  if (a.slots) {
    slot = __builtin_amdgcn_readfirstlane(a.slots[b]);
    int before = 0;
    for (int j = threadIdx.x; j < b; j += kStepThreads) before |= a.slots[j] == slot;
    if (__syncthreads_or(before)) return;
  }
  if (slot < 0 || slot >= a.n_states) return;
  const int64_t at = (static_cast<int64_t>(slot) * a.H + h) * a.dk * a.dv + col;
  float S[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = r * kStepRuns + run;
    S[r] = row < a.dk && col < a.dv ? a.s[at + static_cast<int64_t>(row) * a.dv] : 0.0f;
  }
  auto token = [&](int64_t row) {
    if (threadIdx.x < kStepRuns * NR) {
      ks[threadIdx.x] = kx;
      qs[threadIdx.x] = qx;
    }
    const float decay = a.gate ? exp2_(log2_decay(z, a.gate_kind)) : 1.0f;
    const float eta = a.lr_max / (1.0f + __expf(-(bt + a.lr_bias))), v = vt;
    __syncthreads();
    float e = 0.0f, kq = 0.0f, o = 0.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float kr = ks[r * kStepRuns + run], qr = qs[r * kStepRuns + run];
      S[r] *= decay;
      e += kr * S[r];
      o += qr * S[r];
      kq += kr * qr;
    }
    part[0][run][c] = e;
    part[1][run][c] = o;
    if (c == 0) kq_part[run] = kq;
    __syncthreads();
    e = v;
    o = kq = 0.0f;
#pragma unroll
    for (int j = 0; j < kStepRuns; ++j) {
      e -= part[0][j][c];
      o += part[1][j][c];
      kq += kq_part[j];
    }
    const float u = eta * e;
#pragma unroll
    for (int r = 0; r < NR; ++r) S[r] += ks[r * kStepRuns + run] * u;
    // o = S^T q = (the decayed state)^T q + (k.q) u
    if (run == 0 && col < a.dv) Elem<E>::st(static_cast<E*>(a.o), (row * a.H + h) * a.dv + col, a.scale * (o + kq * u));
    __syncthreads();
  };
  token(b);
  if (a.slots) {
    for (int j0 = b + 1; j0 < a.B; j0 += kStepThreads) {
      const int j = j0 + threadIdx.x;
      const uint64_t hit = __ballot(j < a.B && a.slots[j] == slot);
      if ((threadIdx.x & 63) == 0) same[threadIdx.x >> 6] = hit;
      __syncthreads();
      for (int w = 0; w < kStepThreads / 64; ++w)
        for (uint64_t left = same[w]; left; left &= left - 1) {
          const int row = j0 + w * 64 + __builtin_ctzll(left);
          fetch(row);
          token(row);
        }
      __syncthreads();
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = r * kStepRuns + run;
    if (row < a.dk && col < a.dv) a.s_new[at + static_cast<int64_t>(row) * a.dv] = S[r];
  }
}

template <typename F> hipError_t by_width(int dk, F&& f) {
  if (dk <= 64) return f(std::integral_constant<int, 64>{});
  if (dk <= 128) return f(std::integral_constant<int, 128>{});
  return f(std::integral_constant<int, 256>{});
}

}  // namespace

template <typename E, int DKP, bool BWD> hipError_t launch_prep(const Args& a, hipStream_t s) {
  KernelScope scope(TTT_KERNEL_DELTA_PREP, s);
  prep_kernel<E, DKP, BWD><<<static_cast<uint32_t>(a.chunks) * a.H, kPrepThreads, 0, s>>>(a);
  return hipGetLastError();
}
template hipError_t launch_prep<bf16_t, 64, true>(const Args&, hipStream_t);
template hipError_t launch_prep<bf16_t, 128, true>(const Args&, hipStream_t);
template hipError_t launch_prep<bf16_t, 256, true>(const Args&, hipStream_t);
template hipError_t launch_prep<float, 64, true>(const Args&, hipStream_t);
template hipError_t launch_prep<float, 128, true>(const Args&, hipStream_t);
template hipError_t launch_prep<float, 256, true>(const Args&, hipStream_t);

}  // namespace delta

namespace {

using delta::Args;

int chunk_tokens(int dtype) { return dtype == TTT_F32 ? delta::Chunk<float>::C : delta::Chunk<bf16_t>::C; }
int64_t all_tokens(const ttt_delta_desc& d) { return d.packed ? d.T : static_cast<int64_t>(d.B) * d.T; }
size_t elem_bytes(const ttt_delta_desc& d) { return d.dtype == TTT_F32 ? 4 : 2; }
size_t kept_bytes(const ttt_delta_desc& d) { return d.dtype == TTT_F32 ? delta::kKept<float> : delta::kKept<bf16_t>; }  // of a value for the gradients
int padded_dk(int dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }
size_t tri_bytes(const ttt_delta_desc& d) { return d.dtype == TTT_F32 ? delta::Tri<float>::kBytes : delta::Tri<bf16_t>::kBytes; }

}  // namespace

// Chunk slots: what the sequences take, or for packed ones the most that any lengths take.
int64_t delta_chunks(const ttt_delta_desc& d) {
  const int C = chunk_tokens(d.dtype);
  if (!d.packed) return d.B * ((static_cast<int64_t>(d.T) + C - 1) / C);
  const int64_t n = d.T;
  return n == 0 ? 0 : n / C + (d.B < n ? d.B : n);
}

namespace {

int padded_dv(int dv) { return (dv + 31) / 32 * 32; }

// The pieces of a dense sequence's forward walk, by what a chunk takes: about 2 us with helpers, 2.5 with four
// waves' columns in a workgroup on every CU, 2.2 without outputs, and 2 us more a piece where the maps are joined: figures of
// 128 bf16 channels (2.3, 3.0 and 2.1 at the last measurement) that stand for all widths and both types.  131072 tokens of 16 heads of
// 128: one piece 5.21 ms, four 2.62, eight, which this takes, 2.19, sixteen 2.22.
// Measured for 1, 4 and 16 heads of 64, 128 and 256 channels, bf16 and fp32, at 24, 64, 256 and 1024 chunks: where this cuts, the
// forward takes 0.08 to 0.80 of one piece's time, and up to 1.17 times the best number's; where it does not, 24 chunks would
// take down to 1/1.55 in eight pieces, and 16 heads of 256 at 64 and 256 chunks down to 1/1.6 in four.
int pieces(const ttt_delta_desc& d) {
  if (d.packed || d.T == 0 || d.B == 0) return 1;
  const int64_t chunks = (d.T + chunk_tokens(d.dtype) - 1) / chunk_tokens(d.dtype), heads = static_cast<int64_t>(d.B) * d.H;
  const int64_t gv = (padded_dv(d.dv) + 63) / 64, gm = (padded_dv(d.dv) + padded_dk(d.dk) + 63) / 64;
  if (heads * gv * 2 >= 256) return 1;  // every CU has a walk with helpers
  double best = chunks * 2.0;
  int n = 1;
  for (int64_t k = 2; k <= 64 && 4 * k <= chunks; ++k) {
    const int64_t each = (chunks + k - 1) / k, k1 = (chunks + each - 1) / each;
    const double t = (heads * (k1 - 1) * gm + 255) / 256 * each * 2.2 + k1 * 2.0 + 20.0 + (heads * k1 * gv + 255) / 256 * each * 2.5;
    if (t < (n == 1 ? 0.8 : 1.0) * best) {
      best = t;
      n = static_cast<int>(k1);
    }
  }
  return n;
}

struct Layout {
  size_t edge, base, order, table, vec, t, p, kq, y, after, maps, states, bytes;
};
Layout ws_layout(const ttt_delta_desc& d, bool bwd) {
  const size_t items = static_cast<size_t>(delta_chunks(d)) * d.H, C = chunk_tokens(d.dtype), e = elem_bytes(d);
  const size_t dvp = (d.dv + 31) / 32 * 32;
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += align256(bytes);
    return was;
  };
  if (d.packed && items > 0) {
    l.edge = take(sizeof(int) * (static_cast<size_t>(d.B) + 1));
    l.base = take(sizeof(int) * (static_cast<size_t>(d.B) + 1));
    l.order = take(sizeof(int) * (static_cast<size_t>(d.B) + 1));
    l.table = take(sizeof(int4) * static_cast<size_t>(delta_chunks(d)));
  }
  l.vec = take(items * 3 * C * sizeof(float));
  l.t = take(items * tri_bytes(d));
  l.p = take(items * tri_bytes(d));
  l.kq = take(static_cast<size_t>(delta_chunks(d)) * d.Hk * 2 * C * padded_dk(d.dk) * e);
  if (!bwd && pieces(d) > 1) {
    const size_t all = static_cast<size_t>(d.B) * pieces(d) * d.H * sizeof(float);
    l.maps = take(all * padded_dk(d.dk) * (dvp + padded_dk(d.dk)));
    l.states = take(all * d.dk * d.dv);
  }
  if (bwd) {
    l.y = take(items * C * dvp * kept_bytes(d));
    l.after = take(items * padded_dk(d.dk) * dvp * kept_bytes(d));
  }
  l.bytes = at;
  return l;
}

Args make_args(const ttt_delta_desc& d, const void* q, const void* k, const void* v, const void* gate, const void* beta, const void* d_o) {
  Args a{};
  a.B = d.B; a.T = d.T; a.H = d.H; a.Hk = d.Hk; a.dk = d.dk; a.dv = d.dv;
  a.dvp = (d.dv + 31) / 32 * 32;
  a.packed = d.packed; a.gate_kind = d.gate;
  a.scale = d.scale; a.lr_max = d.lr_max; a.lr_bias = d.lr_bias;
  a.n = all_tokens(d);
  a.ldq = d.ldq ? d.ldq : static_cast<int64_t>(d.Hk) * d.dk;
  a.ldk = d.ldk ? d.ldk : static_cast<int64_t>(d.Hk) * d.dk;
  a.ldv = d.ldv ? d.ldv : static_cast<int64_t>(d.H) * d.dv;
  a.ldg = d.ldg ? d.ldg : d.H;
  a.ldb = d.ldb ? d.ldb : d.H;
  const int V = 16 / static_cast<int>(elem_bytes(d));
  auto wide = [&](const void* p, int width, int64_t ld) {
    return width % V == 0 && ld % V == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  a.q = q; a.k = k; a.v = v; a.gate = gate; a.beta = beta; a.d_o = d_o;
  a.wide_q = wide(q, d.dk, a.ldq);
  a.wide_k = wide(k, d.dk, a.ldk);
  a.wide_v = wide(v, d.dv, a.ldv);
  a.wide_o = a.wide_do = d.dv % V == 0;  // dense, on 16 bytes
  a.dense = a.wide_q && a.wide_k;
  a.chunks = static_cast<int>(delta_chunks(d));
  a.nseg = 1;
  a.seg_chunks = d.packed ? 0 : (d.T + chunk_tokens(d.dtype) - 1) / chunk_tokens(d.dtype);
  a.chunks_per_seq = d.packed ? 0 : (d.T + chunk_tokens(d.dtype) - 1) / chunk_tokens(d.dtype);
  return a;
}

void place(Args& a, const ttt_delta_desc& d, const Layout& l, void* ws, const void* saved) {
  char* w = static_cast<char*>(ws);
  a.vec = reinterpret_cast<float*>(w + l.vec);
  a.t = w + l.t;
  a.p = w + l.p;
  a.kq = w + l.kq;
  a.base = reinterpret_cast<const int*>(w + l.base);
  a.table = reinterpret_cast<const int4*>(w + l.table);
  a.order = reinterpret_cast<const int*>(w + l.order);
  if (saved) {
    const size_t items = static_cast<size_t>(a.chunks) * a.H;
    a.u = const_cast<char*>(static_cast<const char*>(saved));
    a.before = static_cast<char*>(a.u) + align256(items * chunk_tokens(d.dtype) * a.dvp * kept_bytes(d));
  }
}

hipError_t plan(const ttt_delta_desc& d, const Layout& l, const int32_t* starts, void* ws, hipStream_t s) {
  char* w = static_cast<char*>(ws);
  KernelScope scope(TTT_KERNEL_DELTA_PLAN, s);
  delta::plan_kernel<<<1, delta::kPlanThreads, 0, s>>>(starts, d.B, d.T, chunk_tokens(d.dtype), static_cast<int>(delta_chunks(d)),
                                                       reinterpret_cast<int*>(w + l.edge), reinterpret_cast<int*>(w + l.base),
                                                       reinterpret_cast<int4*>(w + l.table), reinterpret_cast<int*>(w + l.order));
  return hipGetLastError();
}

// Without tokens every state passes through.
__global__ void delta_pass_kernel(int64_t n, const float* src, float* dst) {
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) dst[i] = src ? src[i] : 0.0f;
}
hipError_t pass_states(const ttt_delta_desc& d, const float* src, float* dst, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(d.B) * d.H * d.dk * d.dv;
  if (!dst || n == 0) return hipSuccess;
  const int64_t blocks = (n + 255) / 256;
  delta_pass_kernel<<<static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(n, src, dst);
  return hipGetLastError();
}

}  // namespace

size_t delta_workspace(const ttt_delta_desc& d, int entry) {
  return delta_chunks(d) == 0 ? 0 : ws_layout(d, entry == TTT_ENTRY_BWD).bytes;
}
size_t delta_saved(const ttt_delta_desc& d) {
  const size_t items = static_cast<size_t>(delta_chunks(d)) * d.H, e = kept_bytes(d), dvp = (d.dv + 31) / 32 * 32;
  return align256(items * chunk_tokens(d.dtype) * dvp * e) + align256(items * padded_dk(d.dk) * dvp * e);
}

hipError_t delta_fwd_launch(const ttt_delta_desc& d, const void* q, const void* k, const void* v, const void* gate, const void* beta,
                            const float* s0, const int32_t* starts, void* o, float* s_final, void* saved, void* ws, hipStream_t s) {
  Args a = make_args(d, q, k, v, gate, beta, nullptr);
  if (a.n == 0) return pass_states(d, s0, s_final, s);
  a.s0 = s0; a.o = o; a.s_final = s_final;
  const Layout l = ws_layout(d, false);
  place(a, d, l, ws, saved);
  if (d.packed) {
    const hipError_t e = plan(d, l, starts, ws, s);
    if (e != hipSuccess) return e;
  }
  auto run = [&](auto elem, auto width) {
    using E = decltype(elem);
    constexpr int DKP = width();
    hipError_t e = delta::launch_prep<E, DKP, false>(a, s);
    if (e != hipSuccess) return e;
    if (const int n = pieces(d); n > 1) {
      a.nseg = n;
      a.seg_chunks = (a.chunks_per_seq + n - 1) / n;
      float* maps = reinterpret_cast<float*>(static_cast<char*>(ws) + l.maps);
      float* states = reinterpret_cast<float*>(static_cast<char*>(ws) + l.states);
      a.seg_states = states;
      KernelScope scope(TTT_KERNEL_DELTA_MAP, s);
      const int groups = (a.dvp + DKP + 16 * delta::kMapWaves - 1) / (16 * delta::kMapWaves);
      delta::map_kernel<E, DKP><<<delta::walk_grid(a, groups), (delta::kMapWaves + delta::kLoaders) * 64, 0, s>>>(a, groups, maps);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      delta::join_kernel<E, DKP><<<static_cast<uint32_t>(d.B) * d.H * (a.dvp / 16), DKP * 4, 0, s>>>(a, maps, states);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    KernelScope scope(TTT_KERNEL_DELTA_FWD, s);
    return delta::by_waves<DKP>(a, [&](auto waves, int groups) {
      const uint32_t grid = delta::walk_grid(a, groups);
      if (saved) delta::fwd_kernel<E, DKP, waves(), true><<<grid, delta::walk_waves(waves()) * 64, 0, s>>>(a, groups);
      else delta::fwd_kernel<E, DKP, waves(), false><<<grid, delta::walk_waves(waves()) * 64, 0, s>>>(a, groups);
      return hipGetLastError();
    });
  };
  return delta::by_width(d.dk, [&](auto width) { return d.dtype == TTT_F32 ? run(float{}, width) : run(bf16_t{}, width); });
}

hipError_t delta_bwd_launch(const ttt_delta_desc& d, const void* q, const void* k, const void* v, const void* gate, const void* beta,
                            const int32_t* starts, const void* saved, const void* d_o, const float* d_sfinal, void* dq, void* dk,
                            void* dv, void* dgate, void* dbeta, float* ds0, void* ws, hipStream_t s) {
  Args a = make_args(d, q, k, v, gate, beta, d_o);
  if (a.n == 0) return pass_states(d, d_sfinal, ds0, s);
  a.d_sfinal = d_sfinal;
  a.wide_dv = d.dv % (16 / static_cast<int>(elem_bytes(d))) == 0 && a.ldv % (16 / static_cast<int>(elem_bytes(d))) == 0 && reinterpret_cast<uintptr_t>(dv) % 16 == 0;
  a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.dgate = dgate; a.dbeta = dbeta; a.ds0 = ds0;
  const Layout l = ws_layout(d, true);
  place(a, d, l, ws, saved);
  a.y = static_cast<char*>(ws) + l.y;
  a.after = static_cast<char*>(ws) + l.after;
  if (d.packed) {
    const hipError_t e = plan(d, l, starts, ws, s);
    if (e != hipSuccess) return e;
  }
  return delta::by_width(d.dk, [&](auto width) {
    return d.dtype == TTT_F32 ? delta::launch_bwd<float, width()>(a, s) : delta::launch_bwd<bf16_t, width()>(a, s);
  });
}

hipError_t delta_step_launch(const ttt_delta_desc& d, const void* q, const void* k, const void* v, const void* gate, const void* beta,
                             const int32_t* slots, int n_states, const float* st, float* s_new, void* o, hipStream_t s) {
  const Args b = make_args(d, q, k, v, gate, beta, nullptr);
  delta::StepArgs a{d.B, d.H, d.Hk, d.dk, d.dv, d.gate, n_states, (d.dv + delta::kStepCols - 1) / delta::kStepCols,
                    d.scale, d.lr_max, d.lr_bias, b.ldq, b.ldk, b.ldv, b.ldg, b.ldb, q, k, v, gate, beta, slots, st, s_new, o};
  const uint32_t grid = static_cast<uint32_t>(d.B) * d.H * a.ncb;
  KernelScope scope(TTT_KERNEL_DELTA_STEP, s);
  return delta::by_width(d.dk, [&](auto width) {
    constexpr int NR = width() / delta::kStepRuns;
    if (d.dtype == TTT_F32) delta::step_kernel<float, NR><<<grid, delta::kStepThreads, 0, s>>>(a);
    else delta::step_kernel<bf16_t, NR><<<grid, delta::kStepThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace ttt
