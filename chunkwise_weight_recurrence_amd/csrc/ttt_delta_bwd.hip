// Gated delta rule, backward (ttt_delta_common.h has the forward's formulas).  With dO and the gradient dS'
// of the state that leaves a chunk, R_ij = e^{G_i - G_j} and P, T as in the forward:
//   dU = P^T dO + e^{G_C - G} K dS';   Y = T^T dU;   dV = eta Y;
//   dS = e^{G_C} dS' + scale Q^T e^G dO - K^T (e^G eta Y).
// That much is walked through, in the forward's way with everything transposed.  The rest
// is free of it, a chunk a workgroup: with X = scale R o (dO U^T) and M_ij = -eta_i R_ij Y_i.U_j (j < i),
//   dQ = scale e^G dO S^T + X K;
//   dK = [-e^G eta Y S^T + M K] + e^{G_C - G} U dS'^T + X^T Q + M^T K;
//   deta_i = Y_i.e_i, so dbeta_i = (1 - sigmoid) Y_i.U_i.
// Each G_i stands in R, e^G and e^{G_C - G}; what it gathers are row sums that are there already:
//   dG_i = q_i.dq_i - k_i.dk_i + 2 k_i.[...]_i,  and dG_C also e^{G_C} <dS', S> + sum_i e^{G_C - G_i} k_i.(dS' u_i);
// log a_t has the sum of dG_i over i >= t.  Terms that cancel in that sum come from the same rounded X, M, U
// and dS', so they cancel to fp32.

#include "ttt_delta_common.h"

namespace ttt {
namespace delta {
namespace {

// The chain and its helpers where there are few heads, as in the forward.  First half of a chunk: K dS', and by
// the helper P^T dO and scale Q^T e^G dO; second half: Y and the gradient of the state before.  64 chunks of 64 heads
// of 128 bf16 191 us, 208 without helpers.
template <typename E, int DKP, int WAVES, typename Tiles, typename Outs>
__device__ __forceinline__ void help_bwd_or_chain(const Args& a, const Span& span, int seq, int h, int grp, Tiles& tiles, Outs& outs,
                                                  Exchange<E, DKP, WAVES>& exchange) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, ND = DKP / 16, NK = DKP / 32, kMma = sizeof(E) == 2 ? 1 : 4;
  using TR = Tri<E>;
  using Raw = typename Frag<E>::Raw;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const bool helper = threadIdx.x >= WAVES * 64;
  const int wave = (threadIdx.x >> 6) % WAVES, col = (grp * WAVES + wave) * 16 + i;
  char* from_q = exchange.state[wave];
  char* from_p = exchange.rows[wave];
  const int last = span.end - 1;
  if (helper) {
    __syncthreads();
    for (int chunk = last; chunk >= span.first; --chunk) {
      const auto& w = tiles[(last - chunk) & 1];
      Split<E> scores[TR::kFrags];
      f32x4_t go[NT], x[NT], qg[ND], gm[NT];
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) {
        go[mt] = four_of<16 * WAVES>(w.V, 16 * mt + 4 * g, 16 * wave);
        gm[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g);
        x[mt] = zero4();
      }
#pragma unroll
      for (int f = 0; f < TR::kFrags; ++f) scores[f] = tri_load2<E>(w.P, f);
      Raw cols[2][ND];
      auto read_cols = [&](int n) {
#pragma unroll
        for (int t = 0; t < ND; ++t) cols[n & 1][t] = state_col<DKP>(w.Q, 32 * n, t);
      };
      read_cols(0);
      in_order();
#pragma unroll
      for (int kp = 0; kp < NP; ++kp) {
        const Raw e = high(Split<E>(go[2 * kp], go[2 * kp + 1]));  // dO is exact in its type
#pragma unroll
        for (int mt = 0; mt < 2 * kp + 2; ++mt) x[mt] = mma(scores[TR::at_t(mt, kp)], e, x[mt]);
      }
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) go[mt] *= gm[mt] * a.scale;
#pragma unroll
      for (int t = 0; t < ND; ++t) qg[t] = zero4();
      Whole<E> s(go[0], go[1]);
      in_order();
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) give(from_p, mt, x[mt]);
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        if (n + 1 < NP) read_cols(n + 1);
        in_order();
        mma_all(qg, cols[n & 1], s);
        if (n + 1 < NP) s = Whole<E>(go[2 * n + 2], go[2 * n + 3]);
        in_order();
      }
#pragma unroll
      for (int t = 0; t < ND; ++t) give(from_q, t, qg[t]);
      __syncthreads();
      __syncthreads();
    }
    return;
  }
  const bool live = col < a.dvp;
  const int64_t state = (static_cast<int64_t>(seq) * a.H + h) * a.dk * a.dv;
  const uint32_t s_at = col < a.dv ? col * 4 : kNowhere;
  const uint32_t y_at = live ? (col * C + 8 * g) * sizeof(E) : kNowhere, a_at = live ? (col * DKP + 8 * g) * sizeof(E) : kNowhere;
  f32x4_t S[ND];  // dS
  state_load(a.d_sfinal ? a.d_sfinal + state : nullptr, a.dk, a.dv, s_at, S);
  __builtin_amdgcn_s_waitcnt(0);  // here, so that the loop has no wait for memory
  __syncthreads();
  for (int chunk = last; chunk >= span.first; --chunk) {
    const auto& w = tiles[(last - chunk) & 1];
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    const Buffer kept(static_cast<E*>(a.after) + item * a.dvp * DKP, static_cast<int64_t>(a.dvp) * DKP * sizeof(E));
    f32x4_t du[NT], gm[NT], rest[NT], et[NT];
    Raw rows[2][NT];
    auto read_rows = [&](int kp) {
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) rows[kp & 1][mt] = row_frag<DKP>(w.K, 16 * mt + i, 32 * kp + 8 * g);
    };
    Split<E> tri[TR::kFrags];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) du[mt] = zero4();
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
          rest[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + C + 16 * mt + 4 * g);
          et[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 2 * C + 16 * mt + 4 * g);
        }
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) tri[f] = tri_load2<E>(w.T, f);
      }
      kept.store(a_at + 32 * kp * sizeof(E), high(s));
      in_order();
      mma_all(du, rows[kp & 1], s);
      if (kp + 1 < NK) {
        s = Split<E>(S[2 * kp + 2], S[2 * kp + 3]);
        interleave<2 * NT * kMma, 3>();
      }
      in_order();
    }
    const float decay = w.vec[C - 1];
    __syncthreads();
    Raw cols[2][ND];
    auto read_cols = [&](int n) {
#pragma unroll
      for (int t = 0; t < ND; ++t) cols[n & 1][t] = state_col<DKP>(w.K, 32 * n, t);
    };
    f32x4_t y[NT];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      du[mt] = du[mt] * rest[mt] + take(from_p, mt);
      y[mt] = zero4();
    }
    f32x4_t qg[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) qg[t] = take(from_q, t);
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Whole<E> e(du[2 * kp], du[2 * kp + 1]);
      tri_mul<E, true>(y, tri, e, kp);
    }
#pragma unroll
    for (int t = 0; t < ND; ++t) S[t] = S[t] * decay + qg[t];
    in_order();
    read_cols(0);
    const Buffer yb(static_cast<E*>(a.y) + item * a.dvp * C, static_cast<int64_t>(a.dvp) * C * sizeof(E));
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      yb.store(y_at + 32 * kp * sizeof(E), high(Split<E>(y[2 * kp], y[2 * kp + 1])));
#pragma unroll
      for (int mt = 2 * kp; mt < 2 * kp + 2; ++mt) {
        et[mt] *= y[mt];          // dV
        y[mt] = -(gm[mt] * et[mt]);
      }
    }
    Whole<E> x(y[0], y[1]);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      if (n + 1 < NP) read_cols(n + 1);
      in_order();
      mma_all(S, cols[n & 1], x);
      if (n + 1 < NP) x = Whole<E>(y[2 * n + 2], y[2 * n + 3]);
      in_order();
    }
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) out_tile(outs[(last - chunk) & 1], wave, mt, et[mt]);
    __syncthreads();
  }
  if (a.ds0) state_store(a.ds0 + state, a.dk, a.dv, s_at, S);
}

// The walk from the last chunk back, in the forward's way.
template <typename E, int DKP, int WAVES>
__global__ __launch_bounds__(walk_waves(WAVES) * 64, 1) void bwd_kernel(Args a, int groups) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, ND = DKP / 16, NK = DKP / 32, kBuf = kWalkBuffers<E, DKP, WAVES>;
  constexpr int kMma = sizeof(E) == 2 ? 1 : 4;  // matrix instructions of an operand's term
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
    const E* in = static_cast<const E*>(a.d_o) + static_cast<int64_t>(h) * a.dv;
    E* out = static_cast<E*>(a.dv_out) + static_cast<int64_t>(h) * a.dv;
    const int64_t ldo = static_cast<int64_t>(a.H) * a.dv;
    if (a.wide_do && a.wide_dv) load_walk<E, DKP, true, WAVES, kBuf, HELP, true>(a, span, h, grp * WAVES * 16, tiles, outs, in, ldo, out, a.ldv);
    else load_walk<E, DKP, true, WAVES, kBuf, HELP, false>(a, span, h, grp * WAVES * 16, tiles, outs, in, ldo, out, a.ldv);
    return;
  }
  if constexpr (HELP) {
    help_bwd_or_chain<E, DKP, WAVES>(a, span, seq, h, grp, tiles, outs, exchange);
    return;
  }
  const int col = (grp * WAVES + wave) * 16 + i;
  const bool live = col < a.dvp;
  const int64_t state = (static_cast<int64_t>(seq) * a.H + h) * a.dk * a.dv;
  const uint32_t s_at = col < a.dv ? col * 4 : kNowhere;
  f32x4_t S[ND];  // dS
  state_load(a.d_sfinal ? a.d_sfinal + state : nullptr, a.dk, a.dv, s_at, S);
  __builtin_amdgcn_s_waitcnt(0);  // here, so that the loop has no wait for memory
  const uint32_t y_at = live ? (col * C + 8 * g) * sizeof(E) : kNowhere, a_at = live ? (col * DKP + 8 * g) * sizeof(E) : kNowhere;
  const int last = span.end - 1;
  __syncthreads();
  for (int chunk = last; chunk >= span.first; --chunk) {
    const WalkTile<E, DKP, WAVES>& w = tiles[(last - chunk) & (kBuf - 1)];
    OutTile<E, WAVES>& out = outs[(last - chunk) & (kBuf - 1)];
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    // e^{G_C - G} K dS'
    f32x4_t du[NT], go[NT];
    Raw rows[2][NT];
    auto read_rows = [&](int kp) {
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) rows[kp & 1][mt] = row_frag<DKP>(w.K, 16 * mt + i, 32 * kp + 8 * g);
    };
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) du[mt] = zero4();
    read_rows(0);
    Split<E> scores[TR::kFrags], tri[TR::kFrags];
    f32x4_t gm[NT], rest[NT], et[NT];
    const Buffer kept(static_cast<E*>(a.after) + item * a.dvp * DKP, static_cast<int64_t>(a.dvp) * DKP * sizeof(E));
    Split<E> s(S[0], S[1]);
#pragma unroll
    for (int kp = 0; kp < NK; ++kp) {
      if (kp + 1 < NK) {
        read_rows(kp + 1);
      } else {
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
          rest[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + C + 16 * mt + 4 * g);
          go[mt] = four_of<16 * WAVES>(w.V, 16 * mt + 4 * g, 16 * wave);
        }
#pragma unroll
        for (int f = 0; f < TR::kFrags; ++f) scores[f] = tri_load2<E>(w.P, f);
      }
      kept.store(a_at + 32 * kp * sizeof(E), high(s));
      in_order();
      mma_all(du, rows[kp & 1], s);
      if (kp + 1 < NK) {
        s = Split<E>(S[2 * kp + 2], S[2 * kp + 3]);
        interleave<2 * NT * kMma, 3>();
      }
      in_order();
    }
    // + P^T dO (dO is exact in its type)
#pragma unroll
    for (int f = 0; f < TR::kFrags; ++f) tri[f] = tri_load2<E>(w.T, f);
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      gm[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 16 * mt + 4 * g);
      et[mt] = *reinterpret_cast<const f32x4_t*>(w.vec + 2 * C + 16 * mt + 4 * g);
      du[mt] *= rest[mt];
    }
    const float decay = w.vec[C - 1];
    in_order();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Raw e = high(Split<E>(go[2 * kp], go[2 * kp + 1]));
#pragma unroll
      for (int mt = 0; mt < 2 * kp + 2; ++mt) du[mt] = mma(scores[TR::at_t(mt, kp)], e, du[mt]);
    }
#pragma unroll
    for (int t = 0; t < ND; ++t) S[t] *= decay;
    in_order();
    // dS = e^{G_C} dS' + scale Q^T e^G dO - K^T (e^G eta Y), with Y = T^T dU
    Raw cols[2][ND];
    auto read_cols = [&](int n) {  // Q's and K's pairs of token tiles in turn
#pragma unroll
      for (int t = 0; t < ND; ++t) cols[n & 1][t] = state_col<DKP>(n < NP ? w.Q : w.K, 32 * (n % NP), t);
    };
    read_cols(0);
    in_order();
    f32x4_t y[NT];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) y[mt] = zero4();
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      const Whole<E> e(du[2 * kp], du[2 * kp + 1]);
      tri_mul<E, true>(y, tri, e, kp);
    }
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) go[mt] *= gm[mt] * a.scale;
    Whole<E> x(go[0], go[1]);
    in_order();
    const Buffer yb(static_cast<E*>(a.y) + item * a.dvp * C, static_cast<int64_t>(a.dvp) * C * sizeof(E));
    Split<E> ys[NP];
#pragma unroll
    for (int n = 0; n < 2 * NP; ++n) {
      if (n + 1 < 2 * NP) read_cols(n + 1);
      in_order();
      mma_all(S, cols[n & 1], x);
      if (n < NP) {
        ys[n] = Split<E>(y[2 * n], y[2 * n + 1]);
#pragma unroll
        for (int mt = 2 * n; mt < 2 * n + 2; ++mt) {
          et[mt] *= y[mt];          // dV
          y[mt] = -(gm[mt] * et[mt]);
        }
      }
      if (n + 1 < NP) x = Whole<E>(go[2 * n + 2], go[2 * n + 3]);
      else if (n + 1 < 2 * NP) x = Whole<E>(y[2 * (n + 1 - NP)], y[2 * (n + 1 - NP) + 1]);
      interleave<kWhole<E> * ND, 3>();
      in_order();
    }
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) yb.store(y_at + 32 * kp * sizeof(E), high(ys[kp]));
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) out_tile(out, wave, mt, et[mt]);
    if constexpr (kBuf == 1) __syncthreads();
    __syncthreads();
  }
  if (a.ds0) state_store(a.ds0 + state, a.dk, a.dv, s_at, S);
}

// ---- what does not depend on the walk ----

constexpr int kGradThreads = 512, kSlab = 32;  // columns of the values in LDS at a time

template <typename E> __device__ __forceinline__ float dot8(typename Frag<E>::Raw a, typename Frag<E>::Raw b) {
  float s = 0.0f;
  if constexpr (std::is_same_v<E, float>) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s += a.a[j] * b.a[j] + a.b[j] * b.b[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s += from_bf(a[j]) * from_bf(b[j]);
  }
  return s;
}

template <typename E> __device__ __forceinline__ E narrow(float x) {
  if constexpr (std::is_same_v<E, float>) return x;
  else return f32_to_bf16(x);
}

// Four rows r0 .. r0 + 3 of column col0 + i, as a result tile has them.
template <int NCOL> __device__ __forceinline__ f32x4_t four_rows(const bf16_t* lds, int r0, int col0, int tid) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const int i = tid & 15;
  const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + Tile<bf16_t, NCOL>::at(r0 + (i >> 2), col0 + 4 * (i & 3))));
  f32x4_t f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = bf16_to_f32(static_cast<uint16_t>(x[j]));
  return f;
}
template <int NCOL> __device__ __forceinline__ f32x4_t four_rows(const float* lds, int r0, int col0, int tid) {
  f32x4_t f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = lds[Tile<float, NCOL>::at(r0 + j, col0 + (tid & 15))];
  return f;
}

// The sum over 16 lanes, in all of them (rotations within them, without LDS).
__device__ __forceinline__ float sum16(float x) {
#define ROTATED(n) __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x120 + n, 0xf, 0xf, true))
  x += ROTATED(8);
  x += ROTATED(4);
  x += ROTATED(2);
  x += ROTATED(1);
#undef ROTATED
  return x;
}

// The next slab of the values' columns on its way through registers.
template <typename E, int DKP> struct SlabLoader {
  static constexpr int C = Chunk<E>::C, V = 16 / sizeof(E);
  static constexpr int kO = C * kSlab / V, kS = kSlab * DKP / V;  // pieces of dO (and of U, Y); of a state
  static constexpr int nO = (kO + kGradThreads - 1) / kGradThreads, nS = (kS + kGradThreads - 1) / kGradThreads;
  uint4 o[nO], u[nO], y[nO], b[nS], a[nS];
  // Pieces past the end are some thread's twice: both write the same.
  static __device__ __forceinline__ int piece(int n, int all) { return min(static_cast<int>(threadIdx.x) + n * kGradThreads, all - 1); }
  __device__ __forceinline__ void load(const Args& g, int64_t item, const E* dO, int64_t ld, int len, int c0) {
    const int cols = g.dv - c0;  // may be none
    const Buffer ob(dO + c0, cols > 0 ? rows_bytes(len, ld, cols, sizeof(E)) : 0);
    const uint32_t stride = static_cast<uint32_t>(ld * sizeof(E));
    const uint4* up = reinterpret_cast<const uint4*>(static_cast<const E*>(g.u) + (item * g.dvp + c0) * C);
    const uint4* yp = reinterpret_cast<const uint4*>(static_cast<const E*>(g.y) + (item * g.dvp + c0) * C);
    const uint4* bp = reinterpret_cast<const uint4*>(static_cast<const E*>(g.before) + (item * g.dvp + c0) * DKP);
    const uint4* ap = reinterpret_cast<const uint4*>(static_cast<const E*>(g.after) + (item * g.dvp + c0) * DKP);
#pragma unroll
    for (int n = 0; n < nO; ++n) {
      const int x = piece(n, kO), row = x / (kSlab / V), col = x % (kSlab / V) * V;
      if (g.wide_do) {
        o[n] = ob.template load<uint4>(col < cols ? row * stride + col * sizeof(E) : kNowhere);
      } else {
        E e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = ob.template load<E>(col + j < cols ? row * stride + (col + j) * sizeof(E) : kNowhere);
        __builtin_memcpy(&o[n], e, 16);
      }
      u[n] = up[x];
      y[n] = yp[x];
    }
#pragma unroll
    for (int n = 0; n < nS; ++n) {
      b[n] = bp[piece(n, kS)];
      a[n] = ap[piece(n, kS)];
    }
  }
  __device__ __forceinline__ void store(E* dO, E* U, E* Y, E* B, E* A) const {
#pragma unroll
    for (int n = 0; n < nO; ++n) {
      const int x = piece(n, kO);
      *reinterpret_cast<uint4*>(dO + Tile<E, kSlab>::at(x / (kSlab / V), x % (kSlab / V) * V)) = o[n];
      const int at = Tile<E, C>::at(x / (C / V), x % (C / V) * V);
      *reinterpret_cast<uint4*>(U + at) = u[n];
      *reinterpret_cast<uint4*>(Y + at) = y[n];
    }
#pragma unroll
    for (int n = 0; n < nS; ++n) {
      const int x = piece(n, kS), at = Tile<E, DKP>::at(x / (DKP / V), x % (DKP / V) * V);
      *reinterpret_cast<uint4*>(B + at) = b[n];
      *reinterpret_cast<uint4*>(A + at) = a[n];
    }
  }
};

// A chunk and key head a workgroup, the value heads that share it one after the other (SHARED) with dQ and
// dK summed in registers.  Of the triangular products a wave has a row tile of X or of M, of the others an
// eighth of the key channels.  The value columns come 32 at a time.
// Up to 128 bf16 channels two workgroups share a CU (128 registers, 80 KB): 4096 chunks and heads of 128 take 267 us
// so, 317 with one and all in registers.
template <typename E, int DKP, bool SHARED>
__global__ __launch_bounds__(kGradThreads, sizeof(E) == 2 && DKP <= 128 && !SHARED ? 4 : 2) void grad_kernel(Args a) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, NJ = (DKP + 127) / 128, NW = DKP / 16 / NJ;  // NW waves have channels
  using Lds = Tile<E, DKP>;
  using Slab = Tile<E, kSlab>;
  using Sq = Tile<E, C>;
  __shared__ __attribute__((aligned(16))) E K[C * Lds::kRow];
  __shared__ __attribute__((aligned(16))) E Q[C * Lds::kRow];
  __shared__ __attribute__((aligned(16))) E dO[C * Slab::kRow];     // [token][column]
  __shared__ __attribute__((aligned(16))) E U[kSlab * Sq::kRow];    // [column][token]
  __shared__ __attribute__((aligned(16))) E Y[kSlab * Sq::kRow];
  __shared__ __attribute__((aligned(16))) E B[kSlab * Lds::kRow];   // [column][channel]: the state before
  __shared__ __attribute__((aligned(16))) E A[kSlab * Lds::kRow];   // and the gradient of the one after
  __shared__ __attribute__((aligned(16))) E X[C * Sq::kRow];
  __shared__ __attribute__((aligned(16))) E M[C * Sq::kRow];
  __shared__ double G[C];
  __shared__ __attribute__((aligned(16))) float vec[3][C];  // e^G, e^{G_C - G}, eta
  __shared__ float energy[kGradThreads / 64], yu[C];
  float(*sums)[4][C] = reinterpret_cast<float(*)[4][C]>(B);  // [wave], once the slabs are done with
  static_assert(sizeof(float) * NW * 4 * C <= sizeof(B));
  const int chunk = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk, share = a.H / a.Hk;
  const Where w = locate<C>(a, chunk);
  if (w.len < 0) return;
  // lanes are named anew in each stage, so that a stage's LDS addresses do not take registers in the others
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int ch0 = wave * 16 * NJ;  // a wave's first channel
  const bool busy = wave < NW;
  stage<E, C, DKP, kGradThreads>(K, static_cast<const E*>(a.k) + w.token * a.ldk + hk * a.dk, a.ldk, w.len, a.dk, a.wide_k);
  stage<E, C, DKP, kGradThreads>(Q, static_cast<const E*>(a.q) + w.token * a.ldq + hk * a.dk, a.ldq, w.len, a.dk, a.wide_q);
  f32x4_t dq_sum[SHARED ? NT : 1][NJ], dk_sum[SHARED ? NT : 1][NJ];
  if constexpr (SHARED) {
#pragma unroll
    for (int mt = 0; mt < NT; ++mt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) dq_sum[mt][j] = dk_sum[mt][j] = zero4();
  }
  const Buffer qb(static_cast<E*>(a.dq) + w.token * a.ldq + hk * a.dk, rows_bytes(w.len, a.ldq, a.dk, sizeof(E)));
  const Buffer kb(static_cast<E*>(a.dk_out) + w.token * a.ldk + hk * a.dk, rows_bytes(w.len, a.ldk, a.dk, sizeof(E)));
  const uint32_t sq = static_cast<uint32_t>(a.ldq * sizeof(E)), sk = static_cast<uint32_t>(a.ldk * sizeof(E));
  auto store = [&](const f32x4_t& dq, const f32x4_t& dk, int mt, int j) {
    const int i = lane & 15, g = lane >> 4, col = ch0 + 16 * j + i;
    const uint32_t at = busy && col < a.dk ? col * sizeof(E) : kNowhere;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * mt + 4 * g + r;
      qb.store(at + t * sq, narrow<E>(dq[r]));
      kb.store(at + t * sk, narrow<E>(dk[r]));
    }
  };
  // wave w < NT has row tile w of X, wave NT + w that of M
  const int rt = wave % NT;
  const bool tri = wave < 2 * NT, second = wave >= NT;
  for (int hs = 0; hs < (SHARED ? share : 1); ++hs) {
    const int h = hk * share + hs;
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    float sig = 0.0f, z = 0.0f;  // of lane t's token, in wave 0
    __syncthreads();
    if (wave == 0) {
      double Gt;
      float eta;
      gate_lane<E, C>(a, w, h, lane, Gt, eta, sig, z);
      const double last = __shfl(Gt, C - 1, 64);
      if (lane < C) {
        G[lane] = Gt;
        vec[0][lane] = exp2_(static_cast<float>(Gt));
        vec[1][lane] = exp2_(static_cast<float>(last - Gt));
        vec[2][lane] = eta;
      }
    }
    f32x4_t xm[NT], dq[NT][NJ], dkr[NT][NJ], dks[NT][NJ];
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) {
      xm[mt] = zero4();
#pragma unroll
      for (int j = 0; j < NJ; ++j) dq[mt][j] = dkr[mt][j] = dks[mt][j] = zero4();
    }
    float en = 0.0f;
    SlabLoader<E, DKP> slab;
    const E* dop = static_cast<const E*>(a.d_o) + (w.token * a.H + h) * a.dv;
    const int64_t ldo = static_cast<int64_t>(a.H) * a.dv;
    slab.load(a, item, dop, ldo, w.len, 0);
    for (int c0 = 0; c0 < a.dvp; c0 += kSlab) {
      if (c0 > 0) __syncthreads();
      slab.store(dO, U, Y, B, A);
      if (c0 + kSlab < a.dvp) slab.load(a, item, dop, ldo, w.len, c0 + kSlab);
      __syncthreads();
      const int tid = opaque(threadIdx.x), i = tid & 15, g = (tid & 63) >> 4;
      if (tri) {
        const auto x = second ? token_col<C>(Y, rt, tid) : row_frag<kSlab>(dO, 16 * rt + i, 8 * g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xm[nt] = mma(x, token_col<C>(U, nt, tid), xm[nt]);  // those above the diagonal too
      }
      if (busy) {
        typename Frag<E>::Raw sb[NJ], sa[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          sb[j] = plain_col<DKP>(B, 0, ch0 + 16 * j, tid);
          sa[j] = plain_col<DKP>(A, 0, ch0 + 16 * j, tid);
          en += dot8<E>(sb[j], sa[j]);
        }
#pragma unroll
        for (int mt = 0; mt < NT; ++mt) {
          const auto ox = row_frag<kSlab>(dO, 16 * mt + i, 8 * g), ux = token_col<C>(U, mt, tid), yx = token_col<C>(Y, mt, tid);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            dq[mt][j] = mma(ox, sb[j], dq[mt][j]);
            dkr[mt][j] = mma(yx, sb[j], dkr[mt][j]);
            dks[mt][j] = mma(ux, sa[j], dks[mt][j]);
          }
          if (mt % 2) in_order();
        }
      }
    }
    if (tri) {
      const int i = lane & 15, g = lane >> 4;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * rt + 4 * g + r, col = 16 * nt + i;
          const float d = row >= col ? exp2_(static_cast<float>(G[row] - G[col])) : 0.0f;
          if (second) {
            Elem<E>::st(M, Sq::at(row, col), row > col ? -vec[2][row] * d * xm[nt][r] : 0.0f);
            if (row == col) yu[row] = xm[nt][r];
          } else {
            Elem<E>::st(X, Sq::at(row, col), row >= col ? a.scale * d * xm[nt][r] : 0.0f);
          }
        }
    }
    __syncthreads();
    if (busy) {
      const int tid = opaque(threadIdx.x), i = tid & 15, g = (tid & 63) >> 4;
      typename Frag<E>::Raw kc[NJ][NP], qc[NJ][NP];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          kc[j][p] = plain_col<DKP>(K, 32 * p, ch0 + 16 * j, tid);
          qc[j][p] = plain_col<DKP>(Q, 32 * p, ch0 + 16 * j, tid);
        }
#pragma unroll
      for (int mt = 0; mt < NT; ++mt) {
        f32x4_t d1 = zero4(), d2 = zero4(), d3 = zero4(), d4 = zero4();
        const f32x4_t gm = *reinterpret_cast<const f32x4_t*>(&vec[0][16 * mt + 4 * g]);
        const f32x4_t rest = *reinterpret_cast<const f32x4_t*>(&vec[1][16 * mt + 4 * g]);
        const f32x4_t et = *reinterpret_cast<const f32x4_t*>(&vec[2][16 * mt + 4 * g]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int c0 = ch0 + 16 * j;
          dq[mt][j] *= gm * a.scale;
          dkr[mt][j] *= -(gm * et);
          dks[mt][j] *= rest;
#pragma unroll
          for (int p = 0; p <= mt / 2; ++p) {
            dq[mt][j] = mma(row_frag<C>(X, 16 * mt + i, 32 * p + 8 * g), kc[j][p], dq[mt][j]);
            dkr[mt][j] = mma(row_frag<C>(M, 16 * mt + i, 32 * p + 8 * g), kc[j][p], dkr[mt][j]);
          }
          const f32x4_t qv = four_rows<DKP>(Q, 16 * mt + 4 * g, c0, tid), kv = four_rows<DKP>(K, 16 * mt + 4 * g, c0, tid);
          d1 += qv * dq[mt][j];
          d3 += kv * dkr[mt][j];
          d4 += kv * dks[mt][j];
          f32x4_t dk = dkr[mt][j] + dks[mt][j];
#pragma unroll
          for (int p = mt / 2; p < NP; ++p) {
            dk = mma(plain_col<C>(X, 32 * p, 16 * mt, tid), qc[j][p], dk);
            dk = mma(plain_col<C>(M, 32 * p, 16 * mt, tid), kc[j][p], dk);
          }
          d2 += kv * dk;
          if constexpr (SHARED) {
            dq_sum[mt][j] += dq[mt][j];
            dk_sum[mt][j] += dk;
          } else {
            store(dq[mt][j], dk, mt, j);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s1 = sum16(d1[r]), s2 = sum16(d2[r]), s3 = sum16(d3[r]), s4 = sum16(d4[r]);
          if (i == 0) {
            const int t = 16 * mt + 4 * g + r;
            sums[wave][0][t] = s1;
            sums[wave][1][t] = s2;
            sums[wave][2][t] = s3;
            sums[wave][3][t] = s4;
          }
        }
        in_order();
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) en += __shfl_xor(en, d, 64);
    if (lane == 0) energy[wave] = en;
    __syncthreads();
    if (wave == 0) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, all = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        all += energy[v];
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] += lane < C ? sums[v][s][lane] : 0.0f;
      }
      float dG = x[0] - x[1] + 2.0f * x[2], H = x[3];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) H += __shfl_xor(H, d, 64);
#pragma unroll
      for (int d = 1; d < C; d <<= 1) {
        const float o = __shfl_down(dG, d, 64);
        if (lane + d < C) dG += o;
      }
      if (lane < w.len) {
        const int64_t row = w.token + lane;
        Elem<E>::st(static_cast<E*>(a.dbeta), row * a.ldb + h, sig * yu[lane]);
        if (a.dgate) {
          float d = dG + vec[0][C - 1] * all + H;
          if (a.gate_kind == TTT_GATE_SIGMOID) d *= 1.0f / (1.0f + __expf(z));
          if (log2_decay(z, a.gate_kind) <= -150.0f) d = 0.0f;  // the decay itself is zero there
          Elem<E>::st(static_cast<E*>(a.dgate), row * a.ldg + h, d);
        }
      }
    }
  }
  if constexpr (SHARED) {
#pragma unroll
    for (int mt = 0; mt < NT; ++mt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) store(dq_sum[mt][j], dk_sum[mt][j], mt, j);
  }
}

}  // namespace

template <typename E, int DKP> hipError_t launch_bwd(const Args& a, hipStream_t s) {
  hipError_t e = launch_prep<E, DKP, true>(a, s);
  if (e != hipSuccess) return e;
  {
    KernelScope scope(TTT_KERNEL_DELTA_BWD, s);
    e = by_waves<DKP>(a, [&](auto waves, int groups) {
      bwd_kernel<E, DKP, waves()><<<walk_grid(a, groups), walk_waves(waves()) * 64, 0, s>>>(a, groups);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  KernelScope scope(TTT_KERNEL_DELTA_GRAD, s);
  const uint32_t grid = static_cast<uint32_t>(a.chunks) * a.Hk;
  if (a.H == a.Hk) grad_kernel<E, DKP, false><<<grid, kGradThreads, 0, s>>>(a);
  else grad_kernel<E, DKP, true><<<grid, kGradThreads, 0, s>>>(a);
  return hipGetLastError();
}
template hipError_t launch_bwd<bf16_t, 64>(const Args&, hipStream_t);
template hipError_t launch_bwd<bf16_t, 128>(const Args&, hipStream_t);
template hipError_t launch_bwd<bf16_t, 256>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 64>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 128>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 256>(const Args&, hipStream_t);

}  // namespace delta
}  // namespace ttt
