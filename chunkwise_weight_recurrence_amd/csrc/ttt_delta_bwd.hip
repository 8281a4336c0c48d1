// Gated delta rule, backward (ttt_delta_common.h has the forward's formulas).  With dO and the gradient dS'
// of the state that leaves a chunk, R_ij = e^{G_i - G_j} and P, T as in the forward:
//   dU = P^T dO + e^{G_C - G} K dS';   Y = T^T dU;   dV = eta Y;
//   dS = e^{G_C} dS' + scale Q^T e^G dO - K^T (e^G eta Y).
// That much is walked through, in the forward's way with everything transposed.  The rest
// is free of it, a chunk a workgroup, every operand in two bf16 terms or in fp32: with X = scale R o (dO U^T) and M_ij = -eta_i R_ij Y_i.U_j (j < i),
//   dQ = scale e^G dO S^T + X K;
//   dK = [-e^G eta Y S^T + M K] + e^{G_C - G} U dS'^T + X^T Q + M^T K;
//   deta_i = Y_i.e_i, so dbeta_i = (1 - sigmoid) Y_i.U_i.
// Each G_i stands in R, e^G and e^{G_C - G}; what it gathers are row sums that are there already:
//   dG_i = q_i.dq_i - k_i.dk_i + 2 k_i.[...]_i,  and dG_C also e^{G_C} <dS', S> + sum_i e^{G_C - G_i} k_i.(dS' u_i);
// log a_t has the sum of dG_i over i >= t.  Terms that cancel in that sum come from the same X, M, U and dS'.

#include "ttt_delta_common.h"

namespace ttt {
namespace delta {
namespace {

// The chain and its helpers where there are few heads, as in the forward.  First half of a chunk: K dS', and by
// the helper P^T dO and scale Q^T e^G dO; second half: Y and the gradient of the state before.  64 chunks of 64 heads
// of 128 bf16 243 us, with four chain waves a workgroup instead 294.
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
  const uint32_t y_at = live ? (col * C + 8 * g) * kKept<E> : kNowhere, a_at = live ? (col * DKP + 8 * g) * kKept<E> : kNowhere;
  f32x4_t S[ND];  // dS
  state_load(a.d_sfinal ? a.d_sfinal + state : nullptr, a.dk, a.dv, s_at, S);
  __builtin_amdgcn_s_waitcnt(0);  // here, so that the loop has no wait for memory
  __syncthreads();
  for (int chunk = last; chunk >= span.first; --chunk) {
    const auto& w = tiles[(last - chunk) & 1];
    const int64_t item = static_cast<int64_t>(chunk) * a.H + h;
    const Buffer kept(static_cast<char*>(a.after) + item * a.dvp * DKP * kKept<E>, static_cast<int64_t>(a.dvp) * DKP * kKept<E>);
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
      keep<E>(kept, a_at + 32 * kp * kKept<E>, s);
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
    const Buffer yb(static_cast<char*>(a.y) + item * a.dvp * C * kKept<E>, static_cast<int64_t>(a.dvp) * C * kKept<E>);
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) {
      keep<E>(yb, y_at + 32 * kp * kKept<E>, Split<E>(y[2 * kp], y[2 * kp + 1]));
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
  const uint32_t y_at = live ? (col * C + 8 * g) * kKept<E> : kNowhere, a_at = live ? (col * DKP + 8 * g) * kKept<E> : kNowhere;
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
    const Buffer kept(static_cast<char*>(a.after) + item * a.dvp * DKP * kKept<E>, static_cast<int64_t>(a.dvp) * DKP * kKept<E>);
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
      keep<E>(kept, a_at + 32 * kp * kKept<E>, s);
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
    Raw cols[2][TG];
    auto read_cols = [&](int n) {  // Q's and K's pairs of token tiles in turn, each by groups of the state's tiles
      const int q = n / NG;
#pragma unroll
      for (int t = 0; t < TG; ++t) cols[n & 1][t] = state_col<DKP>(q < NP ? w.Q : w.K, 32 * (q % NP), n % NG * TG + t);
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
    const Buffer yb(static_cast<char*>(a.y) + item * a.dvp * C * kKept<E>, static_cast<int64_t>(a.dvp) * C * kKept<E>);
    Split<E> ys[NP];
#pragma unroll
    for (int n = 0; n < 2 * NP * NG; ++n) {
      const int q = n / NG;
      if (n + 1 < 2 * NP * NG) read_cols(n + 1);
      in_order();
      mma_all(tiles_from<TG>(S, n % NG * TG), cols[n & 1], x);
      if (q < NP && n % NG == 0) {
        ys[q] = Split<E>(y[2 * q], y[2 * q + 1]);
#pragma unroll
        for (int mt = 2 * q; mt < 2 * q + 2; ++mt) {
          et[mt] *= y[mt];          // dV
          y[mt] = -(gm[mt] * et[mt]);
        }
      }
      if (n % NG == NG - 1) {
        if (q + 1 < NP) x = Whole<E>(go[2 * q + 2], go[2 * q + 3]);
        else if (q + 1 < 2 * NP) x = Whole<E>(y[2 * (q + 1 - NP)], y[2 * (q + 1 - NP) + 1]);
      }
      interleave<kWhole<E> * TG, 3>();
      in_order();
    }
#pragma unroll
    for (int kp = 0; kp < NP; ++kp) keep<E>(yb, y_at + 32 * kp * kKept<E>, ys[kp]);
#pragma unroll
    for (int mt = 0; mt < NT; ++mt) out_tile(out, wave, mt, et[mt]);
    if constexpr (kBuf == 1) __syncthreads();
    __syncthreads();
  }
  if (a.ds0) state_store(a.ds0 + state, a.dk, a.dv, s_at, S);
}

// ---- what does not depend on the walk ----

constexpr int kSlab = 32;  // columns of the values in LDS at a time
// Sixteen waves, two for each eighth of the key channels with half of the tokens' tiles each, where 128 registers do for
// that (4 x 4096 tokens of 16 heads of 128 bf16, forward and backward, 929 us, 353 of them here; with eight waves 964; heads
// of 64 632 and 647); else eight with 256 registers: with sums of four shared heads 937 (sixteen: 1015), 8 heads of 256 2769 (3311).
template <typename E, int DKP, bool SHARED> constexpr int kHalves = sizeof(E) == 2 && DKP <= 128 && !SHARED ? 2 : 1;
template <typename E, int DKP, bool SHARED> constexpr int kGradThreads = 512 * kHalves<E, DKP, SHARED>;

// An operand in as many terms as are kept, and its products (the smallest first; the product of two second terms is 2^-16 of one).
template <typename E> struct Kept { typename Frag<E>::Raw t[kTerms<E>]; };
template <typename E> __device__ __forceinline__ f32x4_t mma_kept(const Kept<E>& a, typename Frag<E>::Raw b, f32x4_t c) {
#pragma unroll
  for (int n = kTerms<E> - 1; n >= 0; --n) c = mma(a.t[n], b, c);
  return c;
}
template <typename E> __device__ __forceinline__ f32x4_t mma_kept(typename Frag<E>::Raw a, const Kept<E>& b, f32x4_t c) {
#pragma unroll
  for (int n = kTerms<E> - 1; n >= 0; --n) c = mma(a, b.t[n], c);
  return c;
}
template <typename E> __device__ __forceinline__ f32x4_t mma_kept(const Kept<E>& a, const Kept<E>& b, f32x4_t c) {
  if constexpr (kTerms<E> == 2) c = mma(a.t[0], b.t[1], mma(a.t[1], b.t[0], c));
  return mma(a.t[0], b.t[0], c);
}
template <typename E> __device__ __forceinline__ float dot8(const Kept<E>& a, const Kept<E>& b) {
  float s = 0.0f;
  if constexpr (std::is_same_v<E, float>) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s += a.t[0].a[j] * b.t[0].a[j] + a.t[0].b[j] * b.t[0].b[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (from_bf(a.t[0][j]) + from_bf(a.t[1][j])) * (from_bf(b.t[0][j]) + from_bf(b.t[1][j]));
  }
  return s;
}
// A fp32 value's terms, `gap` elements apart.
template <typename E> __device__ __forceinline__ void put_terms(E* p, int at, int gap, float x) {
  Elem<E>::st(p, at, x);
  if constexpr (kTerms<E> == 2) Elem<E>::st(p, at + gap, x - bf16_to_f32(f32_to_bf16(x)));
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

// A workgroup's LDS while the slabs go by, and once they are done with.
template <typename E, int DKP> struct SlabTiles {
  static constexpr int C = Chunk<E>::C, kU = kSlab * Tile<E, C>::kRow, kB = kSlab * Tile<E, DKP>::kRow;  // elements of a term
  E dO[C * Tile<E, kSlab>::kRow];  // [token][column]
  E U[kTerms<E> * kU];             // [term][column][token]
  E Y[kTerms<E> * kU];
  E B[kTerms<E> * kB];             // [term][column][channel]: the state before
  E A[kTerms<E> * kB];             // and the gradient of the one after
};
template <typename E, int NW> struct SquareTiles {
  static constexpr int C = Chunk<E>::C, kX = C * Tile<E, C>::kRow;
  E X[kTerms<E> * kX];
  E M[kTerms<E> * kX];
  float sums[NW][4][C];  // [wave]
};

// The next slab of the values' columns on its way through registers.
template <typename E, int DKP, int THREADS> struct SlabLoader {
  static constexpr int C = Chunk<E>::C, V = 16 / sizeof(E), kThreads = THREADS;
  static constexpr int kO = C * kSlab / V, kU = kTerms<E> * kO, kB = kTerms<E> * kSlab * DKP / V;  // pieces of dO, of U and Y, of the states
  static constexpr int nO = (kO + kThreads - 1) / kThreads, nU = (kU + kThreads - 1) / kThreads, nB = (kB + kThreads - 1) / kThreads;
  typedef uint32_t Vec __attribute__((ext_vector_type(4)));
  Vec o[nO], u[nU], y[nU], b[nB], a[nB];
  // Pieces past the end are some thread's twice: both write the same.
  static __device__ __forceinline__ int piece(int n, int all) { return min(static_cast<int>(threadIdx.x) + n * kThreads, all - 1); }
  __device__ __forceinline__ void load(const Args& g, int64_t item, const E* dO, int64_t ld, int len, int c0) {
    const int cols = g.dv - c0;  // may be none
    const Buffer ob(dO + c0, cols > 0 ? rows_bytes(len, ld, cols, sizeof(E)) : 0);
    const uint32_t stride = static_cast<uint32_t>(ld * sizeof(E));
    const int64_t first = item * g.dvp + c0;  // column
    const Vec* up = reinterpret_cast<const Vec*>(static_cast<const char*>(g.u) + first * C * kKept<E>);
    const Vec* yp = reinterpret_cast<const Vec*>(static_cast<const char*>(g.y) + first * C * kKept<E>);
    const Vec* bp = reinterpret_cast<const Vec*>(static_cast<const char*>(g.before) + first * DKP * kKept<E>);
    const Vec* ap = reinterpret_cast<const Vec*>(static_cast<const char*>(g.after) + first * DKP * kKept<E>);
#pragma unroll
    for (int n = 0; n < nO; ++n) {
      const int x = piece(n, kO), row = x / (kSlab / V), col = x % (kSlab / V) * V;
      if (g.wide_do) {
        o[n] = ob.template load<Vec>(col < cols ? row * stride + col * sizeof(E) : kNowhere);
      } else {
        E e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = ob.template load<E>(col + j < cols ? row * stride + (col + j) * sizeof(E) : kNowhere);
        __builtin_memcpy(&o[n], e, 16);
      }
    }
#pragma unroll
    for (int n = 0; n < nU; ++n) {
      u[n] = up[piece(n, kU)];
      y[n] = yp[piece(n, kU)];
    }
#pragma unroll
    for (int n = 0; n < nB; ++n) {
      b[n] = bp[piece(n, kB)];
      a[n] = ap[piece(n, kB)];
    }
  }
  __device__ __forceinline__ void store(SlabTiles<E, DKP>& s) const {
    using S = SlabTiles<E, DKP>;
#pragma unroll
    for (int n = 0; n < nO; ++n) {
      const int x = piece(n, kO);
      *reinterpret_cast<Vec*>(s.dO + Tile<E, kSlab>::at(x / (kSlab / V), x % (kSlab / V) * V)) = o[n];
    }
#pragma unroll
    for (int n = 0; n < nU; ++n) {
      const int x = piece(n, kU), z = x / kTerms<E>, at = x % kTerms<E> * S::kU + Tile<E, C>::at(z / (C / V), z % (C / V) * V);
      *reinterpret_cast<Vec*>(s.U + at) = u[n];
      *reinterpret_cast<Vec*>(s.Y + at) = y[n];
    }
#pragma unroll
    for (int n = 0; n < nB; ++n) {
      const int x = piece(n, kB), z = x / kTerms<E>, at = x % kTerms<E> * S::kB + Tile<E, DKP>::at(z / (DKP / V), z % (DKP / V) * V);
      *reinterpret_cast<Vec*>(s.B + at) = b[n];
      *reinterpret_cast<Vec*>(s.A + at) = a[n];
    }
  }
};

// The terms of an operand that `read` reads from a tile.
template <typename E, typename F> __device__ __forceinline__ Kept<E> kept(const E* tile, int term, F&& read) {
  Kept<E> k;
#pragma unroll
  for (int n = 0; n < kTerms<E>; ++n) k.t[n] = read(tile + n * term);
  return k;
}

// A chunk and key head a workgroup, the value heads that share it one after the other (SHARED) with dQ and
// dK summed in registers.  Of the triangular products a wave has (half of) a row tile of X or of M, of the others an
// eighth of the key channels, bf16 for half of the tokens.  The value columns come 32 at a time.
template <typename E, int DKP, bool SHARED> __global__ __launch_bounds__((kGradThreads<E, DKP, SHARED>)) void grad_kernel(Args a, int chunk0) {
  constexpr int C = Chunk<E>::C, NT = C / 16, NP = C / 32, NJ = (DKP + 127) / 128, NW = DKP / 16 / NJ;  // NW waves (of a half) have channels
  constexpr int HALVES = kHalves<E, DKP, SHARED>, NH = NT / HALVES, kThreads = kGradThreads<E, DKP, SHARED>;  // token tiles of a wave
  using Lds = Tile<E, DKP>;
  using Sq = Tile<E, C>;
  using Slabs = SlabTiles<E, DKP>;
  using Squares = SquareTiles<E, NW>;
  __shared__ __attribute__((aligned(16))) E K[C * Lds::kRow];
  __shared__ __attribute__((aligned(16))) E Q[C * Lds::kRow];
  __shared__ __attribute__((aligned(16))) char pool[sizeof(Slabs) > sizeof(Squares) ? sizeof(Slabs) : sizeof(Squares)];
  Slabs& s = *reinterpret_cast<Slabs*>(pool);
  Squares& sq = *reinterpret_cast<Squares*>(pool);  // once the slabs are done with
  __shared__ double G[C];
  __shared__ __attribute__((aligned(16))) float vec[3][C];  // e^G, e^{G_C - G}, eta
  __shared__ float energy[NW], yu[C];
  const int chunk = chunk0 + blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk, share = a.H / a.Hk;
  const Where w = locate<C>(a, chunk);
  if (w.len < 0) return;
  // lanes are named anew in each stage, so that a stage's LDS addresses do not take registers in the others
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int ch0 = wave % 8 * 16 * NJ, m0 = wave / 8 * NH;  // a wave's first channel and token tile
  const bool busy = wave % 8 < NW;
  stage<E, C, DKP, kThreads>(K, static_cast<const E*>(a.k) + w.token * a.ldk + hk * a.dk, a.ldk, w.len, a.dk, a.wide_k);
  stage<E, C, DKP, kThreads>(Q, static_cast<const E*>(a.q) + w.token * a.ldq + hk * a.dk, a.ldq, w.len, a.dk, a.wide_q);
  f32x4_t dq_sum[SHARED ? NH : 1][NJ], dk_sum[SHARED ? NH : 1][NJ];
  if constexpr (SHARED) {
#pragma unroll
    for (int m = 0; m < NH; ++m)
#pragma unroll
      for (int j = 0; j < NJ; ++j) dq_sum[m][j] = dk_sum[m][j] = zero4();
  }
  const Buffer qb(static_cast<E*>(a.dq) + w.token * a.ldq + hk * a.dk, rows_bytes(w.len, a.ldq, a.dk, sizeof(E)));
  const Buffer kb(static_cast<E*>(a.dk_out) + w.token * a.ldk + hk * a.dk, rows_bytes(w.len, a.ldk, a.dk, sizeof(E)));
  const uint32_t strideq = static_cast<uint32_t>(a.ldq * sizeof(E)), stridek = static_cast<uint32_t>(a.ldk * sizeof(E));
  auto store = [&](const f32x4_t& dq, const f32x4_t& dk, int mt, int j) {
    const int i = lane & 15, g = lane >> 4, col = ch0 + 16 * j + i;
    const uint32_t at = busy && col < a.dk ? col * sizeof(E) : kNowhere;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * mt + 4 * g + r;
      qb.store(at + t * strideq, narrow<E>(dq[r]));
      kb.store(at + t * stridek, narrow<E>(dk[r]));
    }
  };
  // of the triangular products: whose row tile, and which half of its columns (those above the diagonal are zero)
  const int rt = wave % NT, n0 = wave / NT % HALVES * NH;
  const bool tri = wave < 2 * NT * HALVES, second = wave >= NT * HALVES;
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
    f32x4_t xm[NH], dq[NH][NJ], dkr[NH][NJ], dks[NH][NJ];
#pragma unroll
    for (int m = 0; m < NH; ++m) {
      xm[m] = zero4();
#pragma unroll
      for (int j = 0; j < NJ; ++j) dq[m][j] = dkr[m][j] = dks[m][j] = zero4();
    }
    float en = 0.0f;
    SlabLoader<E, DKP, kThreads> slab;
    const E* dop = static_cast<const E*>(a.d_o) + (w.token * a.H + h) * a.dv;
    const int64_t ldo = static_cast<int64_t>(a.H) * a.dv;
    slab.load(a, item, dop, ldo, w.len, 0);
    for (int c0 = 0; c0 < a.dvp; c0 += kSlab) {
      if (c0 > 0) __syncthreads();
      slab.store(s);
      if (c0 + kSlab < a.dvp) slab.load(a, item, dop, ldo, w.len, c0 + kSlab);
      __syncthreads();
      const int tid = opaque(threadIdx.x), i = tid & 15, g = (tid & 63) >> 4;
      auto tokens = [&](const E* tile, int mt) { return kept<E>(tile, Slabs::kU, [&](const E* t) { return token_col<C>(t, mt, tid); }); };
      if (tri && n0 <= rt) {
        if (second) {
          const auto x = tokens(s.Y, rt);
#pragma unroll
          for (int n = 0; n < NH; ++n) xm[n] = mma_kept<E>(x, tokens(s.U, n0 + n), xm[n]);
        } else {
          const auto x = row_frag<kSlab>(s.dO, 16 * rt + i, 8 * g);
#pragma unroll
          for (int n = 0; n < NH; ++n) xm[n] = mma_kept<E>(x, tokens(s.U, n0 + n), xm[n]);
        }
      }
      if (busy) {
        Kept<E> sb[NJ], sa[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          auto channels = [&](const E* t) { return plain_col<DKP>(t, 0, ch0 + 16 * j, tid); };
          sb[j] = kept<E>(s.B, Slabs::kB, channels);
          sa[j] = kept<E>(s.A, Slabs::kB, channels);
          if (wave < 8) en += dot8<E>(sb[j], sa[j]);
        }
#pragma unroll
        for (int m = 0; m < NH; ++m) {
          const auto ox = row_frag<kSlab>(s.dO, 16 * (m0 + m) + i, 8 * g);
          const auto ux = tokens(s.U, m0 + m), yx = tokens(s.Y, m0 + m);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            dq[m][j] = mma_kept<E>(ox, sb[j], dq[m][j]);
            dkr[m][j] = mma_kept<E>(yx, sb[j], dkr[m][j]);
            dks[m][j] = mma_kept<E>(ux, sa[j], dks[m][j]);
          }
        }
      }
    }
    __syncthreads();
    if (tri) {
      const int i = lane & 15, g = lane >> 4;
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * rt + 4 * g + r, col = 16 * (n0 + n) + i;
          const float d = row >= col ? exp2_(static_cast<float>(G[row] - G[col])) : 0.0f;
          if (second) {
            put_terms<E>(sq.M, Sq::at(row, col), Squares::kX, row > col ? -vec[2][row] * d * xm[n][r] : 0.0f);
            if (row == col) yu[row] = xm[n][r];
          } else {
            put_terms<E>(sq.X, Sq::at(row, col), Squares::kX, row >= col ? a.scale * d * xm[n][r] : 0.0f);
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
      for (int m = 0; m < NH; ++m) {
        const int mt = m0 + m;
        f32x4_t d1 = zero4(), d2 = zero4(), d3 = zero4(), d4 = zero4();
        const f32x4_t gm = *reinterpret_cast<const f32x4_t*>(&vec[0][16 * mt + 4 * g]);
        const f32x4_t rest = *reinterpret_cast<const f32x4_t*>(&vec[1][16 * mt + 4 * g]);
        const f32x4_t et = *reinterpret_cast<const f32x4_t*>(&vec[2][16 * mt + 4 * g]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int c0 = ch0 + 16 * j;
          dq[m][j] *= gm * a.scale;
          dkr[m][j] *= -(gm * et);
          dks[m][j] *= rest;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (p <= mt / 2) {
              auto row = [&](const E* t) { return row_frag<C>(t, 16 * mt + i, 32 * p + 8 * g); };
              dq[m][j] = mma_kept<E>(kept<E>(sq.X, Squares::kX, row), kc[j][p], dq[m][j]);
              dkr[m][j] = mma_kept<E>(kept<E>(sq.M, Squares::kX, row), kc[j][p], dkr[m][j]);
            }
          }
          const f32x4_t qv = four_rows<DKP>(Q, 16 * mt + 4 * g, c0, tid), kv = four_rows<DKP>(K, 16 * mt + 4 * g, c0, tid);
          d1 += qv * dq[m][j];
          d3 += kv * dkr[m][j];
          d4 += kv * dks[m][j];
          f32x4_t dk = dkr[m][j] + dks[m][j];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            if (p >= mt / 2) {
              auto col = [&](const E* t) { return plain_col<C>(t, 32 * p, 16 * mt, tid); };
              dk = mma_kept<E>(kept<E>(sq.X, Squares::kX, col), qc[j][p], dk);
              dk = mma_kept<E>(kept<E>(sq.M, Squares::kX, col), kc[j][p], dk);
            }
          }
          d2 += kv * dk;
          if constexpr (SHARED) {
            dq_sum[m][j] += dq[m][j];
            dk_sum[m][j] += dk;
          } else {
            store(dq[m][j], dk, mt, j);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s1 = sum16(d1[r]), s2 = sum16(d2[r]), s3 = sum16(d3[r]), s4 = sum16(d4[r]);
          if (i == 0) {
            const int t = 16 * mt + 4 * g + r;
            sq.sums[wave % 8][0][t] = s1;
            sq.sums[wave % 8][1][t] = s2;
            sq.sums[wave % 8][2][t] = s3;
            sq.sums[wave % 8][3][t] = s4;
          }
        }
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) en += __shfl_xor(en, d, 64);
    if (lane == 0 && wave < NW) energy[wave] = en;
    __syncthreads();
    if (wave == 0) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, all = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        all += energy[v];
#pragma unroll
        for (int n = 0; n < 4; ++n) x[n] += lane < C ? sq.sums[v][n][lane] : 0.0f;
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
    for (int m = 0; m < NH; ++m)
#pragma unroll
      for (int j = 0; j < NJ; ++j) store(dq_sum[m][j], dk_sum[m][j], m0 + m, j);
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
  auto run = [&](auto shared) {
    constexpr int kThreads = kGradThreads<E, DKP, shared()>;
    const int most = static_cast<int>((UINT32_MAX / kThreads) / a.Hk);  // chunks of a launch, which has fewer than 2^32 threads
    for (int chunk0 = 0; chunk0 < a.chunks; chunk0 += most) {
      const uint32_t grid = static_cast<uint32_t>(a.chunks - chunk0 < most ? a.chunks - chunk0 : most) * a.Hk;
      grad_kernel<E, DKP, shared()><<<grid, kThreads, 0, s>>>(a, chunk0);
      if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  return a.H == a.Hk ? run(std::false_type{}) : run(std::true_type{});
}
template hipError_t launch_bwd<bf16_t, 64>(const Args&, hipStream_t);
template hipError_t launch_bwd<bf16_t, 128>(const Args&, hipStream_t);
template hipError_t launch_bwd<bf16_t, 256>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 64>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 128>(const Args&, hipStream_t);
template hipError_t launch_bwd<float, 256>(const Args&, hipStream_t);

}  // namespace delta
}  // namespace ttt
