// Norm and position rotation of queries and keys on gfx950, one pass over both.
//
// Per token and head, with r = 1 (NONE), (mean(x^2) + eps)^-1/2 (RMS) or (sum(x^2) + eps)^-1/2 (L2):
//   h = r x;  z = w h;  y = z with its first `rot` columns turned pair by pair by pos * inv_freq_j:
//   (z_a, z_b) -> m (z_a cos - z_b sin, z_a sin + z_b cos).
// Backward: dz is dy turned back, dw = sum dz h, dh = w dz,
//   dx = r (dh - h <dh, h>)  (RMS: <dh, h> / D; NONE: dx = dh).
//
// Both directions are bound by HBM.  A token's cosines and sines are formed once for all its
// heads: the angle in 64 bits (position 10^6 times a frequency has no digits left behind the point in 32),
// reduced to half a turn, then the 32-bit functions.  A slot of lanes has one head's row, a lane the
// 16-byte pieces that hold both halves of its pairs, so no lane needs another's values but for the sum.

#include <cstdint>
#include <type_traits>

#include "ttt_device.h"
#include "ttt_internal.h"
#include "ttt_qknorm_unit.h"

namespace ttt {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kFwdGroups = 1 << 20;  // workgroups of the forward, at most
constexpr int kBwdGroups = 1024;  // workgroups of the backward: each writes one partial sum of dw

struct QkArgs {
  int64_t tokens;
  int Hq, Hk, d, rot, norm, period, tok;  // tok: tokens a workgroup takes at a time
  float eps, m;
  int64_t ldq, ldk;
  const void* q;
  const void* k;
  const float* wq;
  const float* wk;
  const int32_t* pos;
  const float* freq;
  void* yq;
  void* yk;
  const void* dyq;
  const void* dyk;
  void* dq;
  void* dk;
  float* part;  // [groups][2][d]
  int want_w;
};

// V elements as they lie.
template <typename E, int V> struct Piece;
template <> struct Piece<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void get(Raw r, float* f) { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
  static __device__ __forceinline__ Raw put(const float* f) { return {f[0], f[1], f[2], f[3]}; }
};
template <> struct Piece<bf16_t, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(Raw r, float* f) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw put(const float* f) {
    return {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
};
template <> struct Piece<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void get(Raw r, float* f) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float* f) { return f[0]; }
};
template <> struct Piece<bf16_t, 1> {
  using Raw = uint16_t;
  static __device__ __forceinline__ void get(Raw r, float* f) { f[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ Raw put(const float* f) { return f32_to_bf16(f[0]); }
};

// The cosines and sines (times m) of `count` tokens, rot / 2 entries a token.
__device__ __forceinline__ void fill_table(float2* table, const QkArgs& a, int64_t t0, int count) {
  const int entries = a.rot / 2;
  for (int x = threadIdx.x; x < count * entries; x += kThreads) {
    const int t = x / entries, j = x % entries;
    const int64_t tok = t0 + t;
    const double p = a.pos ? a.pos[tok] : static_cast<double>(tok % a.period);
    const double turns = p * static_cast<double>(a.freq[j]) * 0.15915494309189533577;
    const float r = static_cast<float>((turns - rint(turns)) * 6.28318530717958647693);
    float s, c;
    sincosf(r, &s, &c);
    table[x] = {a.m * c, a.m * s};
  }
}

// One row's pieces of a lane, turned (BACK: back).  Columns that are in no turned pair are left alone, as are those
// that the row does not have: x cos 0 - y sin 0 is NaN where the neighbour y is infinite.
template <int V, bool HALF, bool BACK>
__device__ __forceinline__ void turn(float (&x)[2][V], const float2* table, const Unit<V, HALF>& u) {
  if constexpr (HALF || V == 1) {
    // V == 1: a pair lies in the two pieces in either order of columns.  All of a unit's pairs are turned or none
    if (u.pairs) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 cs = table[u.t + v];
        const float s = BACK ? -cs.y : cs.y, p = x[0][v], q = x[1][v];
        x[0][v] = p * cs.x - q * s;
        x[1][v] = p * s + q * cs.x;
      }
    }
  } else {
    // selected, not branched over (16384 x 32 rows of 128 bf16, both directions: 144.0 us, 149.1 with a branch a pair)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const int n = (h * V + v) / 2;
        const bool on = n < u.pairs;
        const float2 cs = table[on ? u.t + n : 0];
        const float s = BACK ? -cs.y : cs.y, p = x[h][v], q = x[h][v + 1];
        x[h][v] = on ? p * cs.x - q * s : p;
        x[h][v + 1] = on ? p * s + q * cs.x : q;
      }
  }
}

template <int LANES> __device__ __forceinline__ float slot_sum(float x) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// 1 / size of a row from its sum of squares.
__device__ __forceinline__ float scale_of(const QkArgs& a, float ss) {
  if (a.norm == TTT_HEADNORM_NONE) return 1.0f;
  return 1.0f / sqrtf((a.norm == TTT_HEADNORM_RMS ? ss / a.d : ss) + a.eps);
}

// A unit: 2 V columns; LANES lanes a row, N units a lane.
template <typename E, int V, int LANES, int N, bool HALF>
struct Rows {
  using P = Piece<E, V>;
  using Raw = typename P::Raw;
  static __device__ __forceinline__ void fetch(const E* row, const Unit<V, HALF>& u, int d, Raw (&r)[2]) {
    r[0] = r[1] = Raw{};
    if (u.a < d) r[0] = *reinterpret_cast<const Raw*>(row + u.a);
    if (u.b < d) r[1] = *reinterpret_cast<const Raw*>(row + u.b);
  }
  static __device__ __forceinline__ void load(const E* row, const Unit<V, HALF>& u, int d, float (&x)[2][V]) {
    Raw r[2];
    fetch(row, u, d, r);
    P::get(r[0], x[0]);
    P::get(r[1], x[1]);
  }
  static __device__ __forceinline__ void store(E* row, const Unit<V, HALF>& u, int d, const float (&x)[2][V]) {
    if (u.a < d) *reinterpret_cast<Raw*>(row + u.a) = P::put(x[0]);
    if (u.b < d) *reinterpret_cast<Raw*>(row + u.b) = P::put(x[1]);
  }
  static __device__ __forceinline__ void weights(const float* w, const Unit<V, HALF>& u, int d, float (&x)[2][V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[0][v] = w && u.a < d ? w[u.a + v] : 1.0f;
      x[1][v] = w && u.b < d ? w[u.b + v] : 1.0f;
    }
  }
};

// A slot's rows go over the queries' and the keys' heads of the workgroup's tokens; a row is on its way while the
// one before it (or the table) is computed.  32768 tokens of 40 heads of 128 bf16 (671 MB) 137 us, a copy's rate; 8
// tokens 4.3 us (10.6 with the queries' rows before the keys' and no load ahead).
template <typename E, int V, int LANES, int N, bool HALF>
__global__ __launch_bounds__(kThreads) void qk_fwd_kernel(QkArgs a) {
  using R = Rows<E, V, LANES, N, HALF>;
  extern __shared__ float2 table[];
  constexpr int kSlots = kThreads / LANES;
  const int slot = threadIdx.x / LANES, lane = threadIdx.x % LANES, entries = a.rot / 2, heads = a.Hq + a.Hk;
  float* weights = reinterpret_cast<float*>(table + a.tok * max(entries, 1));  // [2][d]
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok; t0 < a.tokens; t0 += static_cast<int64_t>(gridDim.x) * a.tok) {
    const int count = static_cast<int>(min(static_cast<int64_t>(a.tok), a.tokens - t0)), rows = count * heads;
    typename R::Raw raw[N][2];
    auto fetch = [&](int row) {
      const int t = row / heads, h = row % heads;
      const E* src = h < a.Hq ? static_cast<const E*>(a.q) + (t0 + t) * a.ldq + h * a.d : static_cast<const E*>(a.k) + (t0 + t) * a.ldk + (h - a.Hq) * a.d;
#pragma unroll
      for (int n = 0; n < N; ++n) R::fetch(src, Unit<V, HALF>(lane + n * LANES, a.d, a.rot), a.d, raw[n]);
    };
    if (slot < rows) fetch(slot);
    __syncthreads();
    fill_table(table, a, t0, count);
    for (int x = threadIdx.x; x < 2 * a.d; x += kThreads) {
      const float* w = x < a.d ? a.wq : a.wk;
      weights[x] = w ? w[x < a.d ? x : x - a.d] : 1.0f;
    }
    __syncthreads();
    for (int row = slot; row < rows; row += kSlots) {
      const int t = row / heads, h = row % heads;
      const bool is_q = h < a.Hq;
      const float* w = weights + (is_q ? 0 : a.d);
      float v[N][2][V], ss = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        R::P::get(raw[n][0], v[n][0]);
        R::P::get(raw[n][1], v[n][1]);
#pragma unroll
        for (int j = 0; j < V; ++j) ss += v[n][0][j] * v[n][0][j] + v[n][1][j] * v[n][1][j];
      }
      if (row + kSlots < rows) fetch(row + kSlots);
      const float r = scale_of(a, slot_sum<LANES>(ss));
      E* dst = is_q ? static_cast<E*>(a.yq) + ((t0 + t) * a.Hq + h) * a.d : static_cast<E*>(a.yk) + ((t0 + t) * a.Hk + h - a.Hq) * a.d;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const Unit<V, HALF> u(lane + n * LANES, a.d, a.rot);
        const int pa = min(u.a, a.d - V), pb = min(u.b, a.d - V);  // a piece that is not there takes the last one's
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[n][0][j] *= r * w[pa + j];
          v[n][1][j] *= r * w[pb + j];
        }
        turn<V, HALF, false>(v[n], table + t * entries, u);
        R::store(dst, u, a.d, v[n]);
      }
    }
  }
}

// x is read again and its size formed again, which is free beside the reading.  16384 x 32 rows of 128 bf16 (402 MB)
// 93 us.
template <typename E, int V, int LANES, int N, bool HALF>
__global__ __launch_bounds__(kThreads) void qk_bwd_kernel(QkArgs a) {
  using R = Rows<E, V, LANES, N, HALF>;
  extern __shared__ float2 table[];
  constexpr int kSlots = kThreads / LANES;
  const int slot = threadIdx.x / LANES, lane = threadIdx.x % LANES, entries = a.rot / 2;
  float sum[2][N][2][V] = {};
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok; t0 < a.tokens; t0 += static_cast<int64_t>(gridDim.x) * a.tok) {
    const int count = static_cast<int>(min(static_cast<int64_t>(a.tok), a.tokens - t0));
    __syncthreads();
    fill_table(table, a, t0, count);
    __syncthreads();
    auto part = [&](const E* x, int64_t ld, int H, const float* w, const E* dy, E* dx, float (&dw)[N][2][V]) {
      if (H == 0) return;
      float wv[N][2][V];
#pragma unroll
      for (int n = 0; n < N; ++n) R::weights(w, Unit<V, HALF>(lane + n * LANES, a.d, a.rot), a.d, wv[n]);
      for (int row = slot; row < count * H; row += kSlots) {
        const int t = row / H, h = row % H;
        const int64_t at = (t0 + t) * ld + h * a.d;
        float v[N][2][V], g[N][2][V], ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const Unit<V, HALF> u(lane + n * LANES, a.d, a.rot);
          R::load(x + at, u, a.d, v[n]);
          R::load(dy + ((t0 + t) * H + h) * a.d, u, a.d, g[n]);
#pragma unroll
          for (int j = 0; j < V; ++j) ss += v[n][0][j] * v[n][0][j] + v[n][1][j] * v[n][1][j];
        }
        const float r = scale_of(a, slot_sum<LANES>(ss));
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const Unit<V, HALF> u(lane + n * LANES, a.d, a.rot);
          turn<V, HALF, true>(g[n], table + t * entries, u);
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              v[n][h2][j] *= r;
              dw[n][h2][j] += g[n][h2][j] * v[n][h2][j];
              g[n][h2][j] *= wv[n][h2][j];
              dot += g[n][h2][j] * v[n][h2][j];
            }
        }
        dot = slot_sum<LANES>(dot);
        if (a.norm == TTT_HEADNORM_RMS) dot /= a.d;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const Unit<V, HALF> u(lane + n * LANES, a.d, a.rot);
          if (a.norm != TTT_HEADNORM_NONE) {  // without a norm dx is dh, whatever x is
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
              for (int j = 0; j < V; ++j) g[n][h2][j] = r * (g[n][h2][j] - v[n][h2][j] * dot);
          }
          R::store(dx + at, u, a.d, g[n]);
        }
      }
    };
    part(static_cast<const E*>(a.q), a.ldq, a.Hq, a.wq, static_cast<const E*>(a.dyq), static_cast<E*>(a.dq), sum[0]);
    part(static_cast<const E*>(a.k), a.ldk, a.Hk, a.wk, static_cast<const E*>(a.dyk), static_cast<E*>(a.dk), sum[1]);
  }
  if (!a.want_w) return;
  // the slots' sums, in their order
  __syncthreads();
  float* mine = reinterpret_cast<float*>(table);  // [kSlots][d]
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Unit<V, HALF> u(lane + n * LANES, a.d, a.rot);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (u.a < a.d) mine[slot * a.d + u.a + j] = sum[s][n][0][j];
        if (u.b < a.d) mine[slot * a.d + u.b + j] = sum[s][n][1][j];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kThreads) {
      float x = 0.0f;
      for (int j = 0; j < kSlots; ++j) x += mine[j * a.d + c];
      a.part[(static_cast<int64_t>(blockIdx.x) * 2 + s) * a.d + c] = x;
    }
    __syncthreads();
  }
}

// The workgroups' sums of one column, in a fixed order.
__global__ __launch_bounds__(kThreads) void qk_reduce_kernel(const float* part, int groups, int d, float* dwq, float* dwk) {
  __shared__ float sums[kThreads / 64];
  const int c = blockIdx.x % d, s = blockIdx.x / d;
  float x = 0.0f;
  for (int j = threadIdx.x; j < groups; j += kThreads) x += part[(static_cast<int64_t>(j) * 2 + s) * d + c];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o, 64);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    x = 0.0f;
    for (int j = 0; j < kThreads / 64; ++j) x += sums[j];
    float* dst = s ? dwk : dwq;
    if (dst) dst[c] = x;
  }
}

// ---- host ----

// Whether rows of these tensors and their columns' pairs fall into 16-byte pieces.
bool wide(const ttt_qknorm_desc& d, std::initializer_list<const void*> ptrs) {
  const int V = d.dtype == TTT_F32 ? 4 : 8;
  if (d.d % V || d.ldq % V || d.ldk % V) return false;
  if (d.pairing == TTT_ROPE_HALF && (d.rot / 2 % V || d.rot % V)) return false;
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

// Calls f with the element type, the piece, the lanes of a row and a lane's units as compile-time values.
template <typename F> hipError_t dispatch(const ttt_qknorm_desc& d, bool w, F&& f) {
  auto with = [&](auto e, auto v, auto lanes, auto n) {
    return d.pairing == TTT_ROPE_HALF ? f(e, v, lanes, n, std::true_type{}) : f(e, v, lanes, n, std::false_type{});
  };
  using std::integral_constant;
  auto lanes = [&](auto e, auto v) {
    // the halves' units and the others are counted apart: these may end in half a unit
    const int V = v, nr = d.pairing == TTT_ROPE_HALF ? d.rot / 2 / V : 0;
    const int units = nr + (d.d - 2 * nr * V + 2 * V - 1) / (2 * V);
    if constexpr (v() > 1) {
      if (units <= 4) return with(e, v, integral_constant<int, 4>{}, integral_constant<int, 1>{});
      if (units <= 8) return with(e, v, integral_constant<int, 8>{}, integral_constant<int, 1>{});
      if (units <= 16) return with(e, v, integral_constant<int, 16>{}, integral_constant<int, 1>{});
      // 512 columns are 32 units of 16
      if (v() == 8 || units <= 32) return with(e, v, integral_constant<int, 32>{}, integral_constant<int, 1>{});
      if constexpr (v() < 8) return with(e, v, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    } else {
      if (units <= 64) return with(e, v, integral_constant<int, 64>{}, integral_constant<int, 1>{});
      return with(e, v, integral_constant<int, 64>{}, integral_constant<int, 4>{});
    }
  };
  if (d.dtype == TTT_F32) return w ? lanes(float{}, integral_constant<int, 4>{}) : lanes(float{}, integral_constant<int, 1>{});
  return w ? lanes(bf16_t{}, integral_constant<int, 8>{}) : lanes(bf16_t{}, integral_constant<int, 1>{});
}

QkArgs make_args(const ttt_qknorm_desc& d) {
  QkArgs a{};
  a.tokens = d.tokens; a.Hq = d.Hq; a.Hk = d.Hk; a.d = d.d; a.rot = d.rot; a.norm = d.norm;
  a.period = d.period > 0 ? d.period : INT32_MAX;
  a.eps = d.eps; a.m = d.rot_scale;
  a.ldq = d.ldq ? d.ldq : static_cast<int64_t>(d.Hq) * d.d;
  a.ldk = d.ldk ? d.ldk : static_cast<int64_t>(d.Hk) * d.d;
  // Tokens a workgroup takes: about 256 rows of 128 columns, fewer where that leaves less than 1024 workgroups.  32768
  // tokens of 40 heads of 128 take 139 us forward so, 146 with one token and 144 with four times as many; the
  // backward of 16384 x 32 rows 88, 174 and 94, and 3001 x 6 fp32 rows 12, 13 and 22 forward.
  const int64_t row = static_cast<int64_t>(d.Hq + d.Hk) * d.d;
  int64_t tok = 32768 / row;
  const int64_t share = (d.tokens + 1023) / 1024;
  if (tok > share) tok = share;
  a.tok = static_cast<int>(tok < 1 ? 1 : tok > 16 ? 16 : tok);
  return a;
}
int64_t bwd_groups(const ttt_qknorm_desc& d) {
  const int64_t g = (d.tokens + make_args(d).tok - 1) / make_args(d).tok;
  return g < kBwdGroups ? (g < 1 ? 1 : g) : kBwdGroups;
}
// One entry at least: a pair that is not turned reads the token's first and drops it.
size_t table_bytes(const QkArgs& a) { return static_cast<size_t>(a.tok) * (a.rot > 0 ? a.rot / 2 : 1) * sizeof(float2); }

}  // namespace

size_t qknorm_workspace(const ttt_qknorm_desc& d) { return static_cast<size_t>(bwd_groups(d)) * 2 * d.d * sizeof(float); }

hipError_t qknorm_fwd_launch(const ttt_qknorm_desc& d, const void* q, const void* k, const float* wq, const float* wk,
                             const int32_t* pos, const float* freq, void* yq, void* yk, hipStream_t s) {
  QkArgs a = make_args(d);
  a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.pos = pos; a.freq = freq; a.yq = yq; a.yk = yk;
  return dispatch(d, wide(d, {q, k, yq, yk}), [&](auto e, auto v, auto lanes, auto n, auto half) {
    KernelScope scope(TTT_KERNEL_QK_FWD, s);
    const int64_t groups = (d.tokens + a.tok - 1) / a.tok;
    const uint32_t grid = static_cast<uint32_t>(groups < kFwdGroups ? groups : kFwdGroups);
    qk_fwd_kernel<decltype(e), v(), lanes(), n(), half()><<<grid, kThreads, table_bytes(a) + 2 * d.d * sizeof(float), s>>>(a);
    return hipGetLastError();
  });
}

hipError_t qknorm_bwd_launch(const ttt_qknorm_desc& d, const void* q, const void* k, const float* wq, const float* wk,
                             const int32_t* pos, const float* freq, const void* dyq, const void* dyk, void* dq, void* dk,
                             float* dwq, float* dwk, void* ws, hipStream_t s) {
  QkArgs a = make_args(d);
  a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.pos = pos; a.freq = freq; a.dyq = dyq; a.dyk = dyk; a.dq = dq; a.dk = dk;
  a.part = static_cast<float*>(ws);
  a.want_w = dwq || dwk;
  const int groups = static_cast<int>(bwd_groups(d));
  const hipError_t e0 = dispatch(d, wide(d, {q, k, dyq, dyk, dq, dk}), [&](auto e, auto v, auto lanes, auto n, auto half) {
    KernelScope scope(TTT_KERNEL_QK_BWD, s);
    size_t lds = table_bytes(a);
    const size_t sums = a.want_w ? static_cast<size_t>(kThreads / lanes()) * d.d * sizeof(float) : 0;
    if (lds < sums) lds = sums;
    qk_bwd_kernel<decltype(e), v(), lanes(), n(), half()><<<groups, kThreads, lds, s>>>(a);
    return hipGetLastError();
  });
  if (e0 != hipSuccess || !a.want_w) return e0;
  KernelScope scope(TTT_KERNEL_QK_REDUCE, s);
  qk_reduce_kernel<<<2 * d.d, kThreads, 0, s>>>(a.part, groups, d.d, dwq, dwk);
  return hipGetLastError();
}

}  // namespace ttt
