// Gated linear recurrence on gfx950: per channel, h_t = a_t h_{t-1} + u_t.
//
//   a_t = sigmoid(z_t) or exp(z_t);  u_t = x_t or (1 - a_t) x_t.
// Backward, with e_t the gradient that reaches h_{t-1}:
//   dh_t = do_t + e_{t+1},  e_t = a_t dh_t,
//   dx_t = dh_t (1 or 1 - a_t),  dz_t = dh_t a'_t (h_{t-1} - (0 or x_t)),
// a' = a (1 - a) or a.  Both directions are first-order recurrences, so a run
// of tokens acts on the value that enters it as an affine map v -> A v + B and
// runs compose: that is what splits the token axis.
//
// All sequences lie behind one another on one token axis (a dense [B,T,D] is the
// packed case with a start every T tokens).  A tile is kTile tokens x 64 V
// channels; a wave holds kLW tokens of it in registers, V channels a lane, and
// the waves' maps meet in LDS.  Tiles meet through `agg`, the map of every
// (tile, channel).  A sequence start inside a tile makes its map independent of
// what enters it, so a tile reads the maps back to the tile where the sequence
// of its first token starts, and no further.  Starts are the same for every
// channel, so all control flow on them is wave-uniform.  The state of another
// sequence is never multiplied in (not even by zero): a NaN or an infinity stays
// in its sequence.

#include <cstdint>
#include <type_traits>

#include "ttt_device.h"
#include "ttt_internal.h"

namespace ttt {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kLW = 16;              // tokens a wave holds
constexpr int kTile = kWaves * kLW;  // tokens of a tile

struct RecArgs {
  int B, T, n, D;  // sequences, tokens of each (dense), tokens on the axis, channels
  int nt, ncb, Dp; // tiles, channel blocks, channels rounded up to whole blocks
  int64_t ldx, ldg;
  const int32_t* starts;  // [B + 1], or NULL: a start every T tokens
  const void* x;
  const void* g;
  const float* h0;
  void* o;
  float* h_final;
  float* ckpt;  // [nt][Dp]: the state that enters each tile
  float2* agg;  // [nt][Dp]: each tile's map (A, B)
  const void* d_o;
  const float* d_hfinal;
  void* dx;
  void* dg;
  float* dh0;
};

// V elements of a row, as they lie.
template <typename E, int V> struct Io;
template <> struct Io<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void get(Raw r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};
template <> struct Io<bf16_t, 1> {
  using Raw = uint16_t;
  static __device__ __forceinline__ void get(Raw r, float (&f)[1]) { f[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f32_to_bf16(f[0]); }
};
template <> struct Io<bf16_t, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void get(Raw r, float (&f)[2]) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw put(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
};

// The element at channel c of row t: the row's address is the same for the
// whole wave, the lane adds a 32-bit offset.
template <typename Raw> __device__ __forceinline__ Raw load_at(const void* base, int64_t row_bytes, uint32_t off) {
  return *reinterpret_cast<const Raw*>(static_cast<const char*>(base) + row_bytes + off);
}
template <typename Raw> __device__ __forceinline__ void store_at(void* base, int64_t row_bytes, uint32_t off, Raw v) {
  *reinterpret_cast<Raw*>(static_cast<char*>(base) + row_bytes + off) = v;
}

// a of a gate value.
template <int GATE> __device__ __forceinline__ float gate_a(float z) {
  if constexpr (GATE == TTT_GATE_SIGMOID) return sigmoidf_(z);
  return __expf(z);
}
// 1 - a without the cancellation of the difference: sigmoid: e^-z sigmoid(z)
// (1 where e^-z would pass the range); exp: near 0 the series of 1 - e^z, whose
// first term left out is below 2^-26 of the sum at |z| = 1/2.
template <int GATE> __device__ __forceinline__ float gate_rest(float z, float a) {
  if constexpr (GATE == TTT_GATE_SIGMOID) return z < -80.0f ? 1.0f : __expf(-z) * a;
  float p = 1.0f / 9.0f;
#pragma unroll
  for (int k = 8; k >= 2; --k) p = (1.0f + z * p) * (1.0f / k);
  // now p = (1 + z/3 (1 + z/4 (...))) / 2
  const float s = -z * (1.0f + z * p);
  return fabsf(z) <= 0.5f ? s : 1.0f - a;
}

// What a tile's tokens belong to.  start[j] / end[j]: the sequence that begins /
// ends at the tile's token j, or -1.  Tokens outside lo .. hi - 1 belong to no
// sequence.  first: where the sequence of the tile's first token starts; last:
// where that of its last token ends.  Every value is clamped to the tile or to
// 0 .. n - 1, whatever `starts` holds.
struct Meta {
  int start[kTile], end[kTile];
  int lo, hi, first, last;
};

// The largest j in 0 .. count - 1 with p[j] <= t, or -1 (p sorted); 64 probes a
// step, the result uniform over the wave.
__device__ __forceinline__ int last_not_above(const int32_t* p, int count, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = count;
  while (true) {
    const int step = (n + 63) / 64;
    const int j = lane * step;
    const bool in = j < n && p[lo + j] <= t;
    const int c = __popcll(__ballot(in));
    if (c == 0) return lo - 1;
    lo += (c - 1) * step;
    if (step == 1) return lo;
    n = min(step, n - (c - 1) * step);
  }
}

__device__ __forceinline__ void tile_meta(const RecArgs& a, int t0, Meta& m) {
  const int tid = threadIdx.x;
  const int tl = t0 + kTile - 1;
  if (!a.starts) {
    if (tid < kTile) {
      const int t = t0 + tid;
      int s = -1, e = -1;
      if (t < a.n) {
        const int b = t / a.T, r = t - b * a.T;
        if (r == 0) s = b;
        if (r == a.T - 1) e = b;
      }
      m.start[tid] = s;
      m.end[tid] = e;
    }
    if (tid == 0) {
      m.lo = t0;
      m.hi = min(t0 + kTile, a.n);
      m.first = t0 < a.n ? t0 - t0 % a.T : t0;
      m.last = tl < a.n ? tl - tl % a.T + a.T - 1 : tl;
    }
  } else {
    if (tid < kTile) m.start[tid] = m.end[tid] = -1;
    __syncthreads();
    const int s0 = max(last_not_above(a.starts, a.B + 1, t0), 0);
    for (int j = s0 + tid; j < a.B; j += kThreads) {
      const int p = a.starts[j], q = a.starts[j + 1];
      if (p > tl) break;
      if (q <= p) continue;
      if (p >= t0) m.start[p - t0] = j;
      if (q > t0 && q - 1 <= tl) m.end[q - 1 - t0] = j;
    }
    const int sl = last_not_above(a.starts, a.B + 1, tl);
    if (tid == 0) {
      m.lo = max(t0, a.starts[0]);
      m.hi = min(min(t0 + kTile, a.n), a.starts[a.B]);
      m.first = min(max(a.starts[s0], 0), t0);
      m.last = sl < 0 || sl >= a.B ? tl : min(max(a.starts[sl + 1] - 1, tl), max(a.n - 1, tl));
    }
  }
  __syncthreads();
}

// Sequences without a token: the state passes through (dst = src, or zero).
// Tile i of the grid takes its share of the sequences, a wave one at a time.
__device__ __forceinline__ void pass_empty(const RecArgs& a, int i, int c, bool in, const float* src, float* dst) {
  if (!dst) return;
  if (!a.starts && a.T > 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s1 = static_cast<int>(static_cast<int64_t>(a.B) * (i + 1) / a.nt);
  for (int s = static_cast<int>(static_cast<int64_t>(a.B) * i / a.nt) + wave; s < s1; s += kWaves) {
    if (a.starts && a.starts[s + 1] > a.starts[s]) continue;
    const int64_t at = static_cast<int64_t>(s) * a.D + c;
    if (in) dst[at] = src ? src[at] : 0.0f;
  }
}

// The value that enters a tile, folded over the maps of `count` tiles, first ..
// first + dir (count - 1).  The first tile's map has a reset in it, so only its B
// counts.  Each wave folds a part, the parts meet in `look`; afterwards every
// wave returns the whole fold.
template <int V>
__device__ __forceinline__ void fold_tiles(const RecArgs& a, int first, int count, int dir, int c, float (&look)[kWaves][2 * V][64],
                                           float (&h)[V]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  if (count <= 0) return;  // the same for the whole workgroup
  const int k0 = static_cast<int>(static_cast<int64_t>(count) * wave / kWaves);
  const int k1 = static_cast<int>(static_cast<int64_t>(count) * (wave + 1) / kWaves);
  float A[V], Bv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, Bv[v] = 0.0f;
  for (int k = k0; k < k1; ++k) {
    const float2* p = a.agg + static_cast<int64_t>(first + dir * k) * a.Dp + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 q = p[v];
      Bv[v] = k == 0 ? q.y : q.x * Bv[v] + q.y;
      A[v] = k == 0 ? 0.0f : q.x * A[v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) look[wave][2 * v][lane] = A[v], look[wave][2 * v + 1][lane] = Bv[v];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = look[w][2 * v][lane] * h[v] + look[w][2 * v + 1][lane];
}

constexpr int kAggregate = 0;  // only the tile's map, to agg
constexpr int kOutput = 1;     // reads the maps, writes the outputs

template <typename E, int V, int GATE, int IN, int MODE>
__global__ __launch_bounds__(kThreads) void rec_fwd_kernel(RecArgs a) {
  using IO = Io<E, V>;
  using Raw = typename IO::Raw;
  __shared__ Meta m;
  __shared__ float part[kWaves][2 * V][64];
  __shared__ float look[kWaves][2 * V][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = blockIdx.x / a.ncb, cb = blockIdx.x % a.ncb;
  const int c = (cb * 64 + lane) * V;
  const bool in = c < a.D;
  const uint32_t cl = in ? c : 0;  // lanes past the last channel read the first and store nothing
  const uint32_t off = cl * sizeof(E);
  const int t0 = i * kTile, tw = t0 + wave * kLW;
  const int64_t rx = a.ldx * static_cast<int64_t>(sizeof(E)), rg = a.ldg * static_cast<int64_t>(sizeof(E));
  const int64_t ro = static_cast<int64_t>(a.D) * sizeof(E);

  Raw xr[kLW], gr[kLW];
  if (a.n > 0) {
#pragma unroll
    for (int j = 0; j < kLW; ++j) {
      const int t = min(tw + j, a.n - 1);
      xr[j] = load_at<Raw>(a.x, t * rx, off);
      gr[j] = load_at<Raw>(a.g, t * rg, off);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kLW; ++j) xr[j] = gr[j] = Raw(0);
  }
  tile_meta(a, t0, m);
  const bool mine = lane < kLW;
  const int t = tw + lane, at = mine ? wave * kLW + lane : 0;
  const bool ok = mine && t >= m.lo && t < m.hi;
  const uint32_t okm = static_cast<uint32_t>(__ballot(ok));
  const uint32_t sm = static_cast<uint32_t>(__ballot(ok && m.start[at] >= 0));
  const uint32_t em = static_cast<uint32_t>(__ballot(ok && m.end[at] >= 0));
  const bool simple = okm == (1u << kLW) - 1 && sm == 0;

  float av[kLW][V], uv[kLW][V];
  float A[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, h[v] = 0.0f;
#pragma unroll
  for (int j = 0; j < kLW; ++j) {
    float x[V], z[V];
    IO::get(xr[j], x);
    IO::get(gr[j], z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      av[j][v] = gate_a<GATE>(z[v]);
      uv[j][v] = IN == TTT_REC_PLAIN ? x[v] : gate_rest<GATE>(z[v], av[j][v]) * x[v];
    }
  }
  auto initial = [&](int j, float (&f)[V]) {  // h0 of the sequence that starts at the wave's token j
    const int s = __builtin_amdgcn_readfirstlane(m.start[wave * kLW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = a.h0 ? a.h0[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };
  if (simple) {
#pragma unroll
    for (int j = 0; j < kLW; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = av[j][v] * h[v] + uv[j][v];
        A[v] *= av[j][v];
      }
  } else {
#pragma unroll
    for (int j = 0; j < kLW; ++j) {
      if (!(okm >> j & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v) av[j][v] = 1.0f, uv[j][v] = 0.0f;
      }
      if (sm >> j & 1) initial(j, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = av[j][v] * h[v] + uv[j][v];
        A[v] *= av[j][v];
      }
    }
    // a start: what enters no longer counts.  The sign of A carries it to the readers of `part`.
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = sm ? -1.0f : A[v];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) part[wave][2 * v][lane] = A[v], part[wave][2 * v + 1][lane] = h[v];
  __syncthreads();

  // fold the maps of waves 0 .. upto - 1 onto h; A: the product, dropped at a start
  auto fold_waves = [&](int upto, float (&hh)[V], float (&AA)[V]) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < upto) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float pa = part[w][2 * v][lane], pb = part[w][2 * v + 1][lane];
          const bool reset = pa < 0.0f;
          hh[v] = reset ? pb : pa * hh[v] + pb;
          AA[v] = reset ? 0.0f : pa * AA[v];
        }
      }
    }
  };
  if constexpr (MODE == kAggregate) {
    if (wave == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) A[v] = 1.0f, h[v] = 0.0f;
      fold_waves(kWaves, h, A);
#pragma unroll
      for (int v = 0; v < V; ++v) a.agg[static_cast<int64_t>(i) * a.Dp + c + v] = make_float2(A[v], h[v]);
    }
  } else {
    const int ts = m.first / kTile;
    fold_tiles<V>(a, ts, m.lo < m.hi ? i - ts : 0, 1, c, look, h);
    if (a.ckpt && wave == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) a.ckpt[static_cast<int64_t>(i) * a.Dp + c + v] = h[v];
    }
    fold_waves(wave, h, A);
    if (simple && em == 0) {
#pragma unroll
      for (int j = 0; j < kLW; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = av[j][v] * h[v] + uv[j][v];
        if (in) store_at<Raw>(a.o, (tw + j) * ro, off, IO::put(h));
      }
    } else {
#pragma unroll
      for (int j = 0; j < kLW; ++j) {
        if (sm >> j & 1) initial(j, h);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = av[j][v] * h[v] + uv[j][v];
        if (in && (okm >> j & 1)) store_at<Raw>(a.o, (tw + j) * ro, off, IO::put(h));
        if (in && a.h_final && (em >> j & 1)) {
          const int s = __builtin_amdgcn_readfirstlane(m.end[wave * kLW + j]);
#pragma unroll
          for (int v = 0; v < V; ++v) a.h_final[static_cast<int64_t>(s) * a.D + c + v] = h[v];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) pass_empty(a, i, c + v, in, a.h0, a.h_final);
  }
}

// The backward: the same tiles, e running from the end.  The tile's states are
// formed again from the state that entered it (ckpt) and the waves' forward maps.
template <typename E, int V, int GATE, int IN, int MODE>
__global__ __launch_bounds__(kThreads) void rec_bwd_kernel(RecArgs a) {
  using IO = Io<E, V>;
  using Raw = typename IO::Raw;
  __shared__ Meta m;
  __shared__ float part[kWaves][2 * V][64];   // forward maps
  __shared__ float rpart[kWaves][2 * V][64];  // maps of e, from the end
  __shared__ float look[kWaves][2 * V][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = blockIdx.x / a.ncb, cb = blockIdx.x % a.ncb;
  const int c = (cb * 64 + lane) * V;
  const bool in = c < a.D;
  const uint32_t cl = in ? c : 0;
  const uint32_t off = cl * sizeof(E);
  const int t0 = i * kTile, tw = t0 + wave * kLW;
  const int64_t rx = a.ldx * static_cast<int64_t>(sizeof(E)), rg = a.ldg * static_cast<int64_t>(sizeof(E));
  const int64_t ro = static_cast<int64_t>(a.D) * sizeof(E);

  Raw xr[kLW], gr[kLW], dr[kLW];
  if (a.n > 0) {
#pragma unroll
    for (int j = 0; j < kLW; ++j) {
      const int t = min(tw + j, a.n - 1);
      gr[j] = load_at<Raw>(a.g, t * rg, off);
      dr[j] = load_at<Raw>(a.d_o, t * ro, off);
      xr[j] = load_at<Raw>(a.x, t * rx, off);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kLW; ++j) xr[j] = gr[j] = dr[j] = Raw(0);
  }
  tile_meta(a, t0, m);
  const bool mine = lane < kLW;
  const int t = tw + lane, at = mine ? wave * kLW + lane : 0;
  const bool ok = mine && t >= m.lo && t < m.hi;
  const uint32_t okm = static_cast<uint32_t>(__ballot(ok));
  const uint32_t sm = static_cast<uint32_t>(__ballot(ok && m.start[at] >= 0));
  const uint32_t em = static_cast<uint32_t>(__ballot(ok && m.end[at] >= 0));
  const bool simple = okm == (1u << kLW) - 1 && (sm | em) == 0;

  float av[kLW][V];
#pragma unroll
  for (int j = 0; j < kLW; ++j) {
    float z[V];
    IO::get(gr[j], z);
#pragma unroll
    for (int v = 0; v < V; ++v) av[j][v] = gate_a<GATE>(z[v]);
  }
  // u_t, and 1 - a_t where the input is scaled by it
  auto input = [&](int j, float (&u)[V], float (&rest)[V], float (&x)[V]) {
    float z[V];
    IO::get(xr[j], x);
    IO::get(gr[j], z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      rest[v] = IN == TTT_REC_CONVEX || GATE == TTT_GATE_SIGMOID ? gate_rest<GATE>(z[v], av[j][v]) : 0.0f;
      u[v] = IN == TTT_REC_PLAIN ? x[v] : rest[v] * x[v];
    }
  };
  auto initial = [&](int j, float (&f)[V]) {
    const int s = __builtin_amdgcn_readfirstlane(m.start[wave * kLW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = a.h0 ? a.h0[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };
  auto final_grad = [&](int j, float (&f)[V]) {
    const int s = __builtin_amdgcn_readfirstlane(m.end[wave * kLW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = a.d_hfinal ? a.d_hfinal[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };

  // e's map over the wave's tokens
  float A[V], e[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, e[v] = 0.0f;
#pragma unroll
  for (int j = kLW - 1; j >= 0; --j) {
    if (!simple && (em >> j & 1)) final_grad(j, e);
    float d[V];
    IO::get(dr[j], d);
    if (simple || (okm >> j & 1)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        e[v] = av[j][v] * (d[v] + e[v]);
        A[v] *= av[j][v];
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) rpart[wave][2 * v][lane] = em ? -1.0f : A[v], rpart[wave][2 * v + 1][lane] = e[v];

  if constexpr (MODE == kOutput) {
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, h[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < kLW; ++j) {
      if (!simple && (sm >> j & 1)) initial(j, h);
      float u[V], rest[V], x[V];
      input(j, u, rest, x);
      if (simple || (okm >> j & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[v] = av[j][v] * h[v] + u[v];
          A[v] *= av[j][v];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) part[wave][2 * v][lane] = sm ? -1.0f : A[v], part[wave][2 * v + 1][lane] = h[v];
  }
  __syncthreads();

  if constexpr (MODE == kAggregate) {
    if (wave == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float AA = 1.0f, ee = 0.0f;
#pragma unroll
        for (int w = kWaves - 1; w >= 0; --w) {
          const float pa = rpart[w][2 * v][lane], pb = rpart[w][2 * v + 1][lane];
          ee = pa < 0.0f ? pb : pa * ee + pb;
          AA = pa < 0.0f ? 0.0f : pa * AA;
        }
        a.agg[static_cast<int64_t>(i) * a.Dp + c + v] = make_float2(AA, ee);
      }
    }
  } else {
    // h_{t-1} of every token, kept as w_t = a'_t (h_{t-1} - (0 or x_t))
    float wv[kLW][V];
    {
      float h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = a.ckpt[static_cast<int64_t>(i) * a.Dp + c + v];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float pa = part[w][2 * v][lane], pb = part[w][2 * v + 1][lane];
            h[v] = pa < 0.0f ? pb : pa * h[v] + pb;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kLW; ++j) {
        if (!simple && (sm >> j & 1)) initial(j, h);
        float u[V], rest[V], x[V];
        input(j, u, rest, x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float da = GATE == TTT_GATE_SIGMOID ? av[j][v] * rest[v] : av[j][v];
          wv[j][v] = da * (IN == TTT_REC_PLAIN ? h[v] : h[v] - x[v]);
        }
        if (simple || (okm >> j & 1)) {
#pragma unroll
          for (int v = 0; v < V; ++v) h[v] = av[j][v] * h[v] + u[v];
        }
      }
    }
    const int te = m.last / kTile;
    fold_tiles<V>(a, te, m.lo < m.hi ? te - i : 0, -1, c, look, e);
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w) {
      if (w > wave) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float pa = rpart[w][2 * v][lane], pb = rpart[w][2 * v + 1][lane];
          e[v] = pa < 0.0f ? pb : pa * e[v] + pb;
        }
      }
    }
#pragma unroll
    for (int j = kLW - 1; j >= 0; --j) {
      if (!simple && (em >> j & 1)) final_grad(j, e);
      if (simple || (okm >> j & 1)) {
        float d[V], ox[V], og[V], u[V], rest[V], x[V];
        IO::get(dr[j], d);
        if constexpr (IN == TTT_REC_CONVEX) input(j, u, rest, x);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float dh = d[v] + e[v];
          ox[v] = IN == TTT_REC_PLAIN ? dh : dh * rest[v];
          og[v] = dh * wv[j][v];
          e[v] = av[j][v] * dh;
        }
        if (in) {
          store_at<Raw>(a.dx, (tw + j) * rx, off, IO::put(ox));
          store_at<Raw>(a.dg, (tw + j) * rg, off, IO::put(og));
        }
      }
      if (!simple && in && a.dh0 && (sm >> j & 1)) {
        const int s = __builtin_amdgcn_readfirstlane(m.start[wave * kLW + j]);
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[static_cast<int64_t>(s) * a.D + c + v] = e[v];
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) pass_empty(a, i, c + v, in, a.d_hfinal, a.dh0);
  }
}

// One token for each row: h[slot] <- a h[slot] + u, o = h[slot].  Rows that name
// one slot are consecutive tokens of it, in row order: the first of them does
// them all, so that the result does not depend on which workgroup comes first.
constexpr int kStepThreads = 256;

struct StepArgs {
  int B, D, n_states, ncb;  // ncb: workgroups of a row
  int64_t ldx, ldg;
  const void* x;
  const void* g;
  const int32_t* slots;
  float* h;
  void* o;
};

template <typename E, int V, int GATE, int IN>
__global__ __launch_bounds__(kStepThreads) void rec_step_kernel(StepArgs a) {
  using IO = Io<E, V>;
  using Raw = typename IO::Raw;
  __shared__ uint64_t same[kStepThreads / 64];
  const int b = blockIdx.x / a.ncb;
  const int c = ((blockIdx.x % a.ncb) * kStepThreads + threadIdx.x) * V;
  const bool in = c < a.D;
  const uint32_t off = (in ? c : 0) * sizeof(E);
  const int64_t rx = a.ldx * static_cast<int64_t>(sizeof(E)), rg = a.ldg * static_cast<int64_t>(sizeof(E));
  Raw xr = load_at<Raw>(a.x, b * rx, off), gr = load_at<Raw>(a.g, b * rg, off);
  int slot = b;
  if (a.slots) {
    slot = __builtin_amdgcn_readfirstlane(a.slots[b]);
    int before = 0;
    for (int j = threadIdx.x; j < b; j += kStepThreads) before |= a.slots[j] == slot;
    if (__syncthreads_or(before)) return;
  }
  if (slot < 0 || slot >= a.n_states) return;
  float* hp = a.h + static_cast<int64_t>(slot) * a.D + (in ? c : 0);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = hp[v];
  auto token = [&](int row) {
    float x[V], z[V];
    IO::get(xr, x);
    IO::get(gr, z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float f = gate_a<GATE>(z[v]);
      h[v] = f * h[v] + (IN == TTT_REC_PLAIN ? x[v] : gate_rest<GATE>(z[v], f) * x[v]);
    }
    if (in) store_at<Raw>(a.o, row * static_cast<int64_t>(a.D) * static_cast<int64_t>(sizeof(E)), off, IO::put(h));
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
          xr = load_at<Raw>(a.x, row * rx, off);
          gr = load_at<Raw>(a.g, row * rg, off);
          token(row);
        }
      __syncthreads();
    }
  }
  if (in) {
#pragma unroll
    for (int v = 0; v < V; ++v) hp[v] = h[v];
  }
}

// ---- host ----

// Channels a lane holds: two bf16 where every row starts on a 4-byte boundary.
int lane_channels(int dtype, int D, int64_t ldx, int64_t ldg) {
  return dtype == TTT_BF16 && D % 2 == 0 && ldx % 2 == 0 && ldg % 2 == 0 ? 2 : 1;
}

// Calls f with the element type, V, gate and input as compile-time values.
template <typename F> hipError_t dispatch(const ttt_rec_desc& d, int V, F&& f) {
  auto with_input = [&](auto e, auto v, auto gate) {
    return d.input == TTT_REC_PLAIN ? f(e, v, gate, std::integral_constant<int, TTT_REC_PLAIN>{})
                                    : f(e, v, gate, std::integral_constant<int, TTT_REC_CONVEX>{});
  };
  auto with_gate = [&](auto e, auto v) {
    return d.gate == TTT_GATE_SIGMOID ? with_input(e, v, std::integral_constant<int, TTT_GATE_SIGMOID>{})
                                      : with_input(e, v, std::integral_constant<int, TTT_GATE_LOG>{});
  };
  if (d.dtype == TTT_F32) return with_gate(float{}, std::integral_constant<int, 1>{});
  if (V == 2) return with_gate(bf16_t{}, std::integral_constant<int, 2>{});
  return with_gate(bf16_t{}, std::integral_constant<int, 1>{});
}

int64_t tokens(const ttt_rec_desc& d) { return d.packed ? d.T : static_cast<int64_t>(d.B) * d.T; }
int64_t tiles(const ttt_rec_desc& d) {
  const int64_t nt = (tokens(d) + kTile - 1) / kTile;
  return nt > 0 ? nt : 1;
}
// Room for either channel block width, 64 and 128.
int64_t padded_channels(const ttt_rec_desc& d) { return (static_cast<int64_t>(d.D) + 127) / 128 * 128; }

RecArgs make_args(const ttt_rec_desc& d, int V) {
  RecArgs a{};
  a.B = d.B;
  a.T = d.T;
  a.n = static_cast<int>(tokens(d));
  a.D = d.D;
  a.nt = static_cast<int>(tiles(d));
  a.ncb = (d.D + 64 * V - 1) / (64 * V);
  a.Dp = static_cast<int>(padded_channels(d));
  a.ldx = d.ldx ? d.ldx : d.D;
  a.ldg = d.ldg ? d.ldg : d.D;
  return a;
}

}  // namespace

bool recurrence_grid_fits(const ttt_rec_desc& d) { return tiles(d) * ((static_cast<int64_t>(d.D) + 63) / 64) < (int64_t{1} << 31); }

size_t recurrence_workspace(const ttt_rec_desc& d) {
  if (tiles(d) == 1) return 0;
  return align256(static_cast<size_t>(tiles(d)) * padded_channels(d) * sizeof(float2));
}
size_t recurrence_saved(const ttt_rec_desc& d) {
  return align256(static_cast<size_t>(tiles(d)) * padded_channels(d) * sizeof(float));
}

hipError_t recurrence_fwd_launch(const ttt_rec_desc& d, const void* x, const void* gate, const float* h0, const int32_t* starts,
                                 void* o, float* h_final, void* saved, void* ws, hipStream_t s) {
  const int V = lane_channels(d.dtype, d.D, d.ldx, d.ldg);
  RecArgs a = make_args(d, V);
  a.x = x; a.g = gate; a.h0 = h0; a.starts = d.packed ? starts : nullptr;
  a.o = o; a.h_final = h_final; a.ckpt = static_cast<float*>(saved); a.agg = static_cast<float2*>(ws);
  return dispatch(d, V, [&](auto e, auto v, auto gk, auto in) {
    using E = decltype(e);
    const dim3 grid(static_cast<uint32_t>(a.nt) * a.ncb);
    if (a.nt > 1) {
      KernelScope scope(TTT_KERNEL_REC_FWD, s);
      rec_fwd_kernel<E, v(), gk(), in(), kAggregate><<<grid, kThreads, 0, s>>>(a);
    }
    {
      KernelScope scope(TTT_KERNEL_REC_FWD, s);
      rec_fwd_kernel<E, v(), gk(), in(), kOutput><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
  });
}

hipError_t recurrence_bwd_launch(const ttt_rec_desc& d, const void* x, const void* gate, const float* h0, const int32_t* starts,
                                 const void* saved, const void* d_o, const float* d_hfinal, void* dx, void* dgate, float* dh0,
                                 void* ws, hipStream_t s) {
  const int V = lane_channels(d.dtype, d.D, d.ldx, d.ldg);
  RecArgs a = make_args(d, V);
  a.x = x; a.g = gate; a.h0 = h0; a.starts = d.packed ? starts : nullptr;
  a.ckpt = const_cast<float*>(static_cast<const float*>(saved)); a.agg = static_cast<float2*>(ws);
  a.d_o = d_o; a.d_hfinal = d_hfinal; a.dx = dx; a.dg = dgate; a.dh0 = dh0;
  return dispatch(d, V, [&](auto e, auto v, auto gk, auto in) {
    using E = decltype(e);
    const dim3 grid(static_cast<uint32_t>(a.nt) * a.ncb);
    if (a.nt > 1) {
      KernelScope scope(TTT_KERNEL_REC_BWD, s);
      rec_bwd_kernel<E, v(), gk(), in(), kAggregate><<<grid, kThreads, 0, s>>>(a);
    }
    {
      KernelScope scope(TTT_KERNEL_REC_BWD, s);
      rec_bwd_kernel<E, v(), gk(), in(), kOutput><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
  });
}

hipError_t recurrence_step_launch(const ttt_rec_desc& d, const void* x, const void* gate, const int32_t* slots, int n_states,
                                  float* h, void* o, hipStream_t s) {
  const int V = lane_channels(d.dtype, d.D, d.ldx, d.ldg);
  const int ncb = (d.D + kStepThreads * V - 1) / (kStepThreads * V);
  StepArgs a{d.B, d.D, n_states, ncb, d.ldx ? d.ldx : d.D, d.ldg ? d.ldg : d.D, x, gate, slots, h, o};
  return dispatch(d, V, [&](auto e, auto v, auto gk, auto in) {
    using E = decltype(e);
    const dim3 grid(static_cast<uint32_t>(d.B) * ncb);
    KernelScope scope(TTT_KERNEL_REC_STEP, s);
    rec_step_kernel<E, v(), gk(), in()><<<grid, kStepThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace ttt
