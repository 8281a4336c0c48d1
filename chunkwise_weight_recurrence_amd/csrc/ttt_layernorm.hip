// Layer norm over the rows of [rows, D] on gfx950, forward and backward.
//
//   r = x (+ res, rounded to the tensors' type);  mu, s = 1 / sqrt(var + eps);
//   n = (r - mu) s;  y = n w_g + b_g,  g the row's group (a head's weight, say).
// Backward, with t = w_g dy:
//   dx = s (t - mean(t) - n mean(t n)) (+ dr);  dw_g = sum dy n;  db_g = sum dy.
//
// Both passes are bound by memory: a row is read once into registers, a thread
// holding NIT pieces of VEC elements (16 bytes; rows need not be aligned to them,
// and a last piece that would pass the row's end moves back into it, over elements
// that the piece before has too and that count once: both directions of 60000 x 999
// bf16 166 us, element by element 200, and of 1800000 x 33 220 and 600 us).  Narrow
// rows take a part of a wave each, wide rows as many waves as they have pieces
// for.  Measured, where a copy reaches 4.7 to 4.8 TB/s: forward of
// 32768 x 2560 bf16 with a residual (671 MB) 136 us, both directions of 16384 x 2048
// bf16 with one (537 MB) 103 us, of 262144 x 128 in 16 groups (340 MB) 76 us.
// A workgroup holds several rows side by side (slots), walks over rows of one
// group, so that the weights stay in registers, and takes UR rows a slot at a time:
// they share the barriers of a cross-wave sum, and the loads of the next UR are in
// flight meanwhile.  The variance is the mean of (r - mu)^2 in a second sum over the
// registers, exact also where the mean is far larger than the deviation.
//
// dw and db: a thread owns its columns and sums them over its rows in fp32, the
// slots meet in LDS, and the workgroup writes one partial row; ln_reduce_kernel adds
// the partial rows in a fixed order.

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ttt_device.h"
#include "ttt_internal.h"

namespace ttt {
namespace {

constexpr int kMaxWaves = 16;

struct LnArgs {
  int rows, D, G, period;
  int per_group;  // rows of a group
  int slices;     // workgroups of a group
  int wpr;        // waves of a row (wide rows)
  uint32_t magic; // k / period = (k magic >> 32) >> shift for 0 <= k < 2^31, period > 1
  int shift;
  int64_t ldx;
  float eps;
  const void* x;  // backward: the rows that were normalised
  const void* res;
  const float* w;
  const float* b;
  void* y;
  void* r;
  float* mean;
  float* rstd;
  const void* dy;
  const void* dr;
  void* dx;
  float* part;  // [slices][G][2][D]: partial dw, then partial db
};

template <typename E, int VEC> struct Piece;
template <> struct Piece<bf16_t, 8> {
  typedef uint32_t Raw __attribute__((ext_vector_type(4)));
  typedef Raw Stored __attribute__((aligned(2)));  // as it lies in memory
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(r[k] << 16);
      f[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw put(const float (&f)[8]) {
    return Raw{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
};
template <> struct Piece<float, 4> {
  typedef float Raw __attribute__((ext_vector_type(4)));
  typedef Raw Stored __attribute__((aligned(4)));
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = r[k];
  }
  static __device__ __forceinline__ Raw put(const float (&f)[4]) { return Raw{f[0], f[1], f[2], f[3]}; }
};
template <> struct Piece<bf16_t, 1> {
  using Raw = uint16_t;
  using Stored = uint16_t;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) { f[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f32_to_bf16(f[0]); }
};
template <> struct Piece<float, 1> {
  using Raw = float;
  using Stored = float;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};

// The k-th row of group g.
__device__ __forceinline__ int64_t row_of(const LnArgs& a, int g, int k) {
  if (a.G == 1) return k;
  const int q = a.period == 1 ? k : static_cast<int>(__umulhi(static_cast<uint32_t>(k), a.magic) >> a.shift);
  return (q * a.G + g) * a.period + (k - q * a.period);  // below rows, so below 2^31
}

// v plus the value of the lane that CTRL names in the same 16 lanes.
template <int CTRL> __device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// The sum over each aligned group of LANES lanes, in every lane of it.
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
  v = add_dpp<0xB1>(v);                             // lanes 0 1 | 2 3
  v = add_dpp<0x4E>(v);                             // 0 .. 3
  v = add_dpp<0x141>(v);                            // 0 .. 7, mirrored
  if constexpr (LANES >= 16) v = add_dpp<0x140>(v); // 0 .. 15, mirrored
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (LANES >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// The sum of N values over the TPR lanes of a row (TPR <= 64), or over the `waves`
// waves of a row (TPR == 0, through `lds`, which alternates between two halves so
// that one barrier a call is enough).  Every thread gets the sum; the order is fixed.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int waves, float* lds, int& half) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lanes_sum<TPR ? TPR : 64>(v[k]);
  if constexpr (TPR == 0) {
    if (waves > 1) {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), first = wave / waves * waves;
      float* p = lds + half * N * kMaxWaves;
      half ^= 1;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k * kMaxWaves + wave] = v[k];
      }
      __syncthreads();
      // at most 16 waves: 16 lanes read one value each and add them up
      const int w = threadIdx.x & 15;
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = lanes_sum<16>(w < waves ? p[k * kMaxWaves + first + w] : 0.0f);
    }
  }
}

// The same value, of which the compiler knows nothing: what was formed from it
// before is formed again, not kept in registers.
template <typename Raw> __device__ __forceinline__ Raw afresh(Raw r) {
  if constexpr (sizeof(Raw) == 2) {
    uint32_t q = r;
    asm volatile("" : "+v"(q));
    return static_cast<Raw>(q);
  } else {
    asm volatile("" : "+v"(r));
    return r;
  }
}

// Where a thread stands: its slot, its place in the row and the row's pieces.
template <int VEC, int TPR, int NIT> struct Place {
  int tpr, slots, slot, tr;
  int col[NIT];   // first column of each piece, 0 where it has none
  bool has[NIT];
  int twice[NIT];  // elements at the piece's front that the piece before has too
  __device__ __forceinline__ explicit Place(const LnArgs& a) {
    tpr = TPR ? TPR : a.wpr * 64;
    slots = static_cast<int>(blockDim.x) / tpr;
    slot = threadIdx.x / tpr;
    tr = threadIdx.x - slot * tpr;
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      const int c = (i * tpr + tr) * VEC;
      has[i] = i < NIT - 1 || c < a.D;  // a thread's pieces but the last are whole
      col[i] = has[i] ? min(c, a.D - VEC) : 0;
      twice[i] = i == NIT - 1 && has[i] ? c - col[i] : 0;
    }
  }
  // v where this thread is the one that counts the element, else 0, also where v is
  // no number
  __device__ __forceinline__ float once(int i, int e, float v) const { return i < NIT - 1 || (has[i] && e >= twice[i]) ? v : 0.0f; }
};

// UR rows of a slot as they lie in memory, NT tensors of them.
template <typename E, int VEC, int TPR, int NIT, int UR, int NT> struct Batch {
  using Raw = typename Piece<E, VEC>::Raw;
  Raw r[NT][UR][NIT];
  int64_t row[UR];
  bool ok[UR];
  __device__ __forceinline__ void rows(const LnArgs& a, const Place<VEC, TPR, NIT>& at, int g, int64_t k0) {
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int64_t k = k0 + u * at.slots + at.slot;
      ok[u] = k < a.per_group;
      row[u] = row_of(a, g, static_cast<int>(ok[u] ? k : 0));
    }
  }
  __device__ __forceinline__ void load(int n, const void* base, int64_t ld, const Place<VEC, TPR, NIT>& at) {
#pragma unroll
    for (int u = 0; u < UR; ++u)
#pragma unroll
      for (int i = 0; i < NIT; ++i) r[n][u][i] = *reinterpret_cast<const typename Piece<E, VEC>::Stored*>(static_cast<const E*>(base) + row[u] * ld + at.col[i]);
  }
};

// A workgroup's size at most.
constexpr int max_threads(int tpr, int ur) { return tpr ? 256 : ur > 1 ? 512 : 1024; }

template <typename E, int VEC, int TPR, int NIT, int UR, bool RES>
__global__ __launch_bounds__(max_threads(TPR, UR)) void ln_fwd_kernel(LnArgs a) {
  using P = Piece<E, VEC>;
  using Raw = typename P::Raw;
  __shared__ float lds[2 * UR * kMaxWaves];
  int half = 0;
  const Place<VEC, TPR, NIT> at(a);
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  float w[NIT][VEC], b[NIT][VEC];
#pragma unroll
  for (int i = 0; i < NIT; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = a.w ? a.w[static_cast<int64_t>(g) * a.D + at.col[i] + e] : 1.0f;
      b[i][e] = a.b ? a.b[static_cast<int64_t>(g) * a.D + at.col[i] + e] : 0.0f;
    }
  const float inv = 1.0f / static_cast<float>(a.D);
  const int64_t step = static_cast<int64_t>(a.slices) * at.slots * UR;
  int64_t k0 = static_cast<int64_t>(slice) * at.slots * UR;
  Batch<E, VEC, TPR, NIT, UR, RES ? 2 : 1> next;
  auto fetch = [&](int64_t k) {
    next.rows(a, at, g, k);
    next.load(0, a.x, a.ldx, at);
    if constexpr (RES) next.load(1, a.res, a.D, at);
  };
  // the next rows' loads are in flight while these are worked on, where the registers allow it
  constexpr bool AHEAD = NIT * VEC <= 8;
  if (AHEAD) fetch(k0);
  for (; k0 < a.per_group; k0 += step) {
    if (!AHEAD) fetch(k0);
    float f[UR][NIT][VEC], sum[UR];
    int64_t row[UR];
    bool ok[UR];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      row[u] = next.row[u];
      ok[u] = next.ok[u];
      sum[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        P::get(next.r[0][u][i], f[u][i]);
        if constexpr (RES) {
          float q[VEC];
          P::get(next.r[1][u][i], q);
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[u][i][e] += q[e];
          // the stream is normalised as it is kept, so that the backward sees the same rows
          P::get(P::put(f[u][i]), f[u][i]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[u] += at.once(i, e, f[u][i][e]);
      }
    }
    if (AHEAD && k0 + step < a.per_group) fetch(k0 + step);
    row_sum<TPR, UR>(sum, a.wpr, lds, half);
    // Kept only now that every thread of the row has read it: r may be res, and pieces
    // overlap.  The rounding is exact, f was rounded before.
    if constexpr (RES) {
#pragma unroll
      for (int u = 0; u < UR; ++u)
#pragma unroll
        for (int i = 0; i < NIT; ++i)
          if (ok[u] && at.has[i])
            *reinterpret_cast<typename P::Stored*>(static_cast<E*>(a.r) + row[u] * a.D + at.col[i]) = P::put(f[u][i]);
    }
    float mu[UR], var[UR];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      mu[u] = sum[u] * inv;
      var[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NIT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          f[u][i][e] -= mu[u];
          var[u] += at.once(i, e, f[u][i][e] * f[u][i][e]);
        }
    }
    row_sum<TPR, UR>(var, a.wpr, lds, half);
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const float s = 1.0f / sqrtf(var[u] * inv + a.eps);
      if (!ok[u]) continue;
      if (at.tr == 0) {
        if (a.mean) a.mean[row[u]] = mu[u];
        if (a.rstd) a.rstd[row[u]] = s;
      }
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = f[u][i][e] * s * w[i][e] + b[i][e];
        if (at.has[i]) *reinterpret_cast<typename P::Stored*>(static_cast<E*>(a.y) + row[u] * a.D + at.col[i]) = P::put(y);
      }
    }
  }
}

template <typename E, int VEC, int TPR, int NIT, int UR, bool RES>
__global__ __launch_bounds__(max_threads(TPR, UR)) void ln_bwd_kernel(LnArgs a) {
  using P = Piece<E, VEC>;
  using Raw = typename P::Raw;
  constexpr int kThreads = max_threads(TPR, UR);
  __shared__ float lds[4 * UR * kMaxWaves];
  __shared__ float cols[NIT == 1 ? kThreads * VEC : 1];  // rows of more pieces are alone in a workgroup
  int half = 0;
  const Place<VEC, TPR, NIT> at(a);
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  // The widest rows leave no registers for the weights, which are read again for each
  // row (from L2), nor, with 24 columns of a thread, for its sums of dw: those lie in LDS.
  constexpr bool KEEP = NIT == 1, FAR = NIT * VEC >= 20;
  __shared__ float4 far[FAR ? NIT * VEC / 4 * kThreads : 1];
  const float* wg = a.w ? a.w + static_cast<int64_t>(g) * a.D : nullptr;
  float w[KEEP ? NIT : 1][VEC], dw[FAR ? 1 : NIT][VEC], db[NIT][VEC];
#pragma unroll
  for (int i = 0; i < NIT; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (KEEP) w[i][e] = wg ? wg[at.col[i] + e] : 1.0f;
      if constexpr (!FAR) dw[i][e] = 0.0f;
      db[i][e] = 0.0f;
    }
  if constexpr (FAR) {
#pragma unroll
    for (int q = 0; q < NIT * VEC / 4; ++q) far[q * kThreads + threadIdx.x] = float4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  auto weights = [&](int i, float (&v)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if constexpr (KEEP) v[e] = w[i][e];
      else v[e] = wg ? wg[at.col[i] + e] : 1.0f;
  };
  const float inv = 1.0f / static_cast<float>(a.D);
  const int64_t step = static_cast<int64_t>(a.slices) * at.slots * UR;
  int64_t k0 = static_cast<int64_t>(slice) * at.slots * UR;
  Batch<E, VEC, TPR, NIT, UR, RES ? 3 : 2> next;
  float mu_next[UR], s_next[UR];
  auto fetch = [&](int64_t k) {
    next.rows(a, at, g, k);
    next.load(0, a.x, a.ldx, at);
    next.load(1, a.dy, a.D, at);
    if constexpr (RES) next.load(2, a.dr, a.D, at);
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      mu_next[u] = a.mean[next.row[u]];
      s_next[u] = a.rstd[next.row[u]];
    }
  };
  constexpr bool AHEAD = NIT * VEC <= 8;
  if (AHEAD && k0 < a.per_group) fetch(k0);
  for (; k0 < a.per_group; k0 += step) {
    if (!AHEAD) fetch(k0);
    const Batch<E, VEC, TPR, NIT, UR, RES ? 3 : 2> cur = next;
    float sum[2 * UR], mu[UR], s[UR];
#pragma unroll
    for (int u = 0; u < UR; ++u) mu[u] = mu_next[u], s[u] = s_next[u];
    if (AHEAD && k0 + step < a.per_group) fetch(k0 + step);
    // n and t = w dy of a piece; formed from the packed rows in both walks
    auto values = [&](int u, int i, float (&n)[VEC], float (&dy)[VEC]) {
      P::get(afresh(cur.r[0][u][i]), n);
      P::get(afresh(cur.r[1][u][i]), dy);
#pragma unroll
      for (int e = 0; e < VEC; ++e) n[e] = (n[e] - mu[u]) * s[u];
    };
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      sum[2 * u] = sum[2 * u + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);  // one piece's weights at a time
        float n[VEC], dy[VEC], wi[VEC];
        values(u, i, n, dy);
        weights(i, wi);
        if constexpr (FAR) {  // one row at a time, which is there
#pragma unroll
          for (int q = 0; q < VEC / 4; ++q) {
            float4& to = far[(i * (VEC / 4) + q) * kThreads + threadIdx.x];
            float4 v = to;
            v.x += dy[4 * q] * n[4 * q];
            v.y += dy[4 * q + 1] * n[4 * q + 1];
            v.z += dy[4 * q + 2] * n[4 * q + 2];
            v.w += dy[4 * q + 3] * n[4 * q + 3];
            to = v;
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if constexpr (!FAR) dw[i][e] += cur.ok[u] ? dy[e] * n[e] : 0.0f;
          db[i][e] += cur.ok[u] ? dy[e] : 0.0f;
          const float t = wi[e] * dy[e];
          sum[2 * u] += at.once(i, e, t);
          sum[2 * u + 1] += at.once(i, e, t * n[e]);
        }
      }
    }
    row_sum<TPR, 2 * UR>(sum, a.wpr, lds, half);
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      if (!cur.ok[u]) continue;
      const float m1 = sum[2 * u] * inv, m2 = sum[2 * u + 1] * inv;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);
        float n[VEC], d[VEC], q[VEC], wi[VEC];
        values(u, i, n, d);
        weights(i, wi);
        if constexpr (RES) P::get(cur.r[2][u][i], q);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          d[e] = s[u] * (wi[e] * d[e] - m1 - n[e] * m2);
          if constexpr (RES) d[e] += q[e];
        }
        E* to = static_cast<E*>(a.dx) + cur.row[u] * a.ldx + at.col[i];
        if (at.twice[i] == 0) {
          if (at.has[i]) *reinterpret_cast<typename P::Stored*>(to) = P::put(d);
        } else {  // one piece of a row: the elements of its own
#pragma unroll
          for (int e = 1; e < VEC; ++e)
            if (e >= at.twice[i]) Elem<E>::st(to, e, d[e]);
        }
      }
    }
  }
  if (!a.part) return;
  // the slots' sums meet in LDS, the first slot's threads add them up
  float* out = a.part + (static_cast<int64_t>(slice) * a.G + g) * 2 * a.D;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      if constexpr (NIT == 1) {
        if (at.slots > 1) {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < VEC; ++e) cols[e * kThreads + threadIdx.x] = which ? db[i][e] : dw[i][e];
          __syncthreads();
        }
      }
      if (at.slot == 0 && at.has[i]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float v;
          if constexpr (FAR) v = which ? db[i][e] : reinterpret_cast<const float*>(&far[(i * (VEC / 4) + e / 4) * kThreads + threadIdx.x])[e % 4];
          else v = which ? db[i][e] : dw[i][e];
          if constexpr (NIT == 1)
            for (int q = 1; q < at.slots; ++q) v += cols[e * kThreads + q * at.tpr + at.tr];
          if (e >= at.twice[i]) out[which * a.D + at.col[i] + e] = v;
        }
      }
    }
  }
}

// Rows that no workgroup holds in registers (see make_plan): every sum walks over the
// row again, which L2 still has by then.  Bound by those walks: 1500 x 32768 bf16 take
// 134 us forward (196 MB, 1.5 TB/s) and 379 backward, where dw and db are read and
// written for every row.
constexpr int kLongThreads = 1024;

template <typename E>
__global__ __launch_bounds__(kLongThreads) void ln_fwd_long_kernel(LnArgs a) {
  __shared__ float lds[2 * kMaxWaves];
  int half = 0;
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  const float* w = a.w ? a.w + static_cast<int64_t>(g) * a.D : nullptr;
  const float* b = a.b ? a.b + static_cast<int64_t>(g) * a.D : nullptr;
  const float inv = 1.0f / static_cast<float>(a.D);
  for (int k = slice; k < a.per_group; k += a.slices) {
    const int64_t row = row_of(a, g, k);
    const E* x = static_cast<const E*>(a.x) + row * a.ldx;
    const E* q = a.res ? static_cast<const E*>(a.res) + row * a.D : nullptr;
    E* r = static_cast<E*>(a.r) + row * a.D;
    E* y = static_cast<E*>(a.y) + row * a.D;
    float sum[1] = {0.0f}, var[1] = {0.0f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      float f = Elem<E>::ld(x, c);
      if (q) {
        Elem<E>::st(r, c, f + Elem<E>::ld(q, c));
        f = Elem<E>::ld(r, c);
      }
      sum[0] += f;
    }
    row_sum<0, 1>(sum, kMaxWaves, lds, half);
    const float mu = sum[0] * inv;
    const E* src = q ? r : x;  // each thread reads the columns that it wrote
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float f = Elem<E>::ld(src, c) - mu;
      var[0] += f * f;
    }
    row_sum<0, 1>(var, kMaxWaves, lds, half);
    const float s = 1.0f / sqrtf(var[0] * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = s;
    }
    for (int c = threadIdx.x; c < a.D; c += kLongThreads)
      Elem<E>::st(y, c, (Elem<E>::ld(src, c) - mu) * s * (w ? w[c] : 1.0f) + (b ? b[c] : 0.0f));
  }
}

template <typename E>
__global__ __launch_bounds__(kLongThreads) void ln_bwd_long_kernel(LnArgs a) {
  __shared__ float lds[4 * kMaxWaves];
  int half = 0;
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  const float* w = a.w ? a.w + static_cast<int64_t>(g) * a.D : nullptr;
  const float inv = 1.0f / static_cast<float>(a.D);
  float* out = a.part ? a.part + (static_cast<int64_t>(slice) * a.G + g) * 2 * a.D : nullptr;
  if (out)
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) out[c] = out[a.D + c] = 0.0f;
  for (int k = slice; k < a.per_group; k += a.slices) {
    const int64_t row = row_of(a, g, k);
    const E* x = static_cast<const E*>(a.x) + row * a.ldx;
    const E* dy = static_cast<const E*>(a.dy) + row * a.D;
    const E* dr = a.dr ? static_cast<const E*>(a.dr) + row * a.D : nullptr;
    E* dx = static_cast<E*>(a.dx) + row * a.ldx;
    const float mu = a.mean[row], s = a.rstd[row];
    float sum[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float d = Elem<E>::ld(dy, c), n = (Elem<E>::ld(x, c) - mu) * s, t = d * (w ? w[c] : 1.0f);
      if (out) {
        out[c] += d * n;
        out[a.D + c] += d;
      }
      sum[0] += t;
      sum[1] += t * n;
    }
    row_sum<0, 2>(sum, kMaxWaves, lds, half);
    const float m1 = sum[0] * inv, m2 = sum[1] * inv;
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float n = (Elem<E>::ld(x, c) - mu) * s, t = Elem<E>::ld(dy, c) * (w ? w[c] : 1.0f);
      Elem<E>::st(dx, c, s * (t - m1 - n * m2) + (dr ? Elem<E>::ld(dr, c) : 0.0f));
    }
  }
}

// dw[g][c], db[g][c] = the sum of their `slices` partial rows: 32 columns a
// workgroup, 32 threads a column, each adds every 32nd partial row.  Bound by latency:
// 5 us for the 4 MB of a training step.
constexpr int kReduceCols = 32, kReduceThreads = 1024, kReduceRows = kReduceThreads / kReduceCols;
constexpr int kReduceGrid = 1 << 20;  // workgroups at most: a launch has fewer than 2^32 threads

__global__ __launch_bounds__(kReduceThreads) void ln_reduce_kernel(const float* __restrict__ part, int slices, int G, int D,
                                                                   float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[kReduceRows][kReduceCols];
  const int lane = threadIdx.x % kReduceCols, row = threadIdx.x / kReduceCols;
  const int64_t cols = static_cast<int64_t>(G) * 2 * D;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kReduceCols; c0 < cols; c0 += static_cast<int64_t>(kReduceGrid) * kReduceCols) {
    const int64_t c = c0 + lane;
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 8
      for (int s = row; s < slices; s += kReduceRows) v += part[s * cols + c];
    }
    sums[row][lane] = v;
    __syncthreads();
    if (row == 0 && c < cols) {
      v = 0.0f;
#pragma unroll
      for (int w = 0; w < kReduceRows; ++w) v += sums[w][lane];
      const int64_t g = c / (2 * D), q = c - g * 2 * D;
      float* to = q < D ? dw : db;
      if (to) to[g * D + (q < D ? q : q - D)] = v;
    }
    __syncthreads();
  }
}

// ---- host ----

// How a row is laid over threads.
struct Plan {
  int vec;      // elements of a piece
  int tpr;      // lanes of a row (8 .. 64), or 0: whole waves
  int nit;      // pieces of a thread; 0: the long kernels
  int wpr;      // waves of a row where tpr is 0
  int slots;    // rows side by side
  int threads;  // of a workgroup
};

constexpr int kWideThreads = 512;  // of a workgroup of wide rows, where one row does not take more

Plan make_plan(const ttt_ln_desc& d) {
  const int wide = d.dtype == TTT_BF16 ? 8 : 4;
  Plan p{};
  p.vec = d.D >= wide ? wide : 1;
  const int pieces = (d.D + p.vec - 1) / p.vec;
  if (pieces <= 64) {
    p.tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    p.nit = 1;
    p.threads = 256;
    p.slots = 256 / p.tpr;
    return p;
  }
  // Pieces of a thread.  More than three of 8 elements (five of 4), held twice in the
  // backward and with their sums, do not fit in a thread's 128 registers; below that they
  // are the faster way, also where the compiler keeps some in scratch: both directions of
  // 3000 x 19992 bf16 242 us, by the long kernels 875.
  constexpr int kAll = kLongThreads;  // a piece each
  p.nit = pieces <= kAll ? 1 : pieces <= 2 * kAll ? 2 : pieces <= 3 * kAll ? 3 : pieces <= 5 * kAll && d.dtype == TTT_F32 ? 5 : 0;
  if (!p.nit) {
    p.slots = 1;
    p.threads = kLongThreads;
    return p;
  }
  p.wpr = ((pieces + p.nit - 1) / p.nit + 63) / 64;
  p.slots = p.wpr * 64 >= kWideThreads ? 1 : kWideThreads / (p.wpr * 64);
  p.threads = p.slots * p.wpr * 64;
  return p;
}

// Workgroups a CU, each of which walks over its share of the rows.  The forward has
// about 1024 lanes a CU that hold a piece: idle lanes do not count, since it is the
// loads in flight that matter.  32768 x 2560 bf16 with a residual takes 136 us (2048
// threads 146), 4000 x 1024 12.7 (18.1), 50000 x 640 39.2 (1024 threads 41.1),
// 7000 x 6000 47.6 (rounded down to one 57.5).  Narrow rows take
// 1024 threads, idle lanes or not: 262144 x 128 29.9 us (2048 threads 31.6), 500000 x 100
// 42.2 (2048 42.7, 1024 lanes with a piece 46.3).  Rows that no workgroup holds: 1500 x 32768
// 135 us with two of 1024 threads, 199 with one.  (These and the figures below: mean device
// time of a launch, other inputs from launch to launch.)
int fwd_per_cu(const ttt_ln_desc& d, const Plan& p) {
  if (p.tpr) return 1024 / p.threads;
  if (!p.nit) return 2;
  const int per = p.vec * p.nit, lanes = p.slots * ((d.D + per - 1) / per);
  return (1024 + lanes - 1) / lanes;
}
// The backward's workgroups each write a partial row of dw and db: 512 threads, one
// workgroup at least.  16384 x 2048 bf16 takes 50 us with 512, 56 with 1024 and 68 with
// 2048, 262144 x 128 41, 47 and 49; 7000 x 8192 81 with one of 1024 threads on every CU,
// 122 on every other.
int bwd_per_cu(const Plan& p) { return std::max(512 / p.threads, 1); }

// Workgroups of each group, no more than there are rows for (`unroll` of them a step).
int slices_of(const ttt_ln_desc& d, const Plan& p, int unroll, int per_cu) {
  const int64_t per_group = d.rows / d.groups;
  const int64_t steps = (per_group + p.slots * unroll - 1) / (p.slots * unroll);
  const int64_t want = (static_cast<int64_t>(256) * per_cu + d.groups - 1) / d.groups;
  const int64_t n = steps < want ? steps : want;
  return static_cast<int>(n > 0 ? n : 1);
}

// Rows a slot takes at once, where there are enough for every workgroup; few rows go
// to as many workgroups as there are.  Wide rows share barriers: forward of 50000 x 640
// bf16 45.6 us with one and 39.2 with two, 16384 x 2048 with a residual 53.6 and 51.0, its
// backward 48.5 and 50.4.  Narrow rows have no barrier to share but short loads: forward of
// 262144 x 128 34.0 us with one, 33.1 with two, 29.9 with four; the backward (registers for
// two tensors more) 45.8, 40.7 and 43.1.
int fwd_unroll(const ttt_ln_desc& d, const Plan& p) {
  if (p.nit != 1 || p.threads > kWideThreads || d.rows < 4096 * p.slots) return 1;
  return p.tpr ? 4 : 2;
}
int bwd_unroll(const ttt_ln_desc& d, const Plan& p) {
  return p.nit != 1 || p.threads > kWideThreads || d.rows < 4096 * p.slots ? 1 : 2;
}

int bwd_slices(const ttt_ln_desc& d) {
  const Plan p = make_plan(d);
  return slices_of(d, p, bwd_unroll(d, p), bwd_per_cu(p));
}

// Calls f with the element type and the plan as compile-time values.
template <bool FWD, typename F> hipError_t dispatch(const ttt_ln_desc& d, const Plan& p, int unroll, bool res, F&& f) {
  auto with_res = [&](auto e, auto vec, auto tpr, auto nit, auto ur) {
    return res ? f(e, vec, tpr, nit, ur, std::true_type{}) : f(e, vec, tpr, nit, ur, std::false_type{});
  };
  auto with_rows = [&](auto e, auto vec, auto tpr, auto nit) {
    if constexpr (nit() == 1) {
      if (unroll > 1) return with_res(e, vec, tpr, nit, std::integral_constant<int, FWD && tpr() != 0 ? 4 : 2>{});
    }
    return with_res(e, vec, tpr, nit, std::integral_constant<int, 1>{});
  };
  auto with_plan = [&](auto e, auto vec) {
    std::integral_constant<int, 1> one;
    if constexpr (vec() == 1) {  // fewer columns than a piece has
      return with_rows(e, vec, std::integral_constant<int, 8>{}, one);
    } else {
      switch (p.tpr) {
        case 8: return with_rows(e, vec, std::integral_constant<int, 8>{}, one);
        case 16: return with_rows(e, vec, std::integral_constant<int, 16>{}, one);
        case 32: return with_rows(e, vec, std::integral_constant<int, 32>{}, one);
        case 64: return with_rows(e, vec, std::integral_constant<int, 64>{}, one);
      }
      std::integral_constant<int, 0> group;
      if constexpr (std::is_same_v<decltype(e), float>) {
        if (p.nit == 5) return with_rows(e, vec, group, std::integral_constant<int, 5>{});
      }
      if (p.nit == 3) return with_rows(e, vec, group, std::integral_constant<int, 3>{});
      if (p.nit == 2) return with_rows(e, vec, group, std::integral_constant<int, 2>{});
      return with_rows(e, vec, group, one);
    }
  };
  auto one = std::integral_constant<int, 1>{};
  if (d.dtype == TTT_BF16) return p.vec == 8 ? with_plan(bf16_t{}, std::integral_constant<int, 8>{}) : with_plan(bf16_t{}, one);
  return p.vec == 4 ? with_plan(float{}, std::integral_constant<int, 4>{}) : with_plan(float{}, one);
}

LnArgs make_args(const ttt_ln_desc& d) {
  LnArgs a{};
  a.rows = static_cast<int>(d.rows);
  a.D = d.D;
  a.G = d.groups;
  a.period = d.period;
  a.per_group = a.rows / a.G;
  // With 2^(s-1) < period <= 2^s, magic = ceil(2^(31+s) / period) is below 2^32 and off
  // by less than 2^s / 2^(31+s) of a quotient's step for every k < 2^31: the floor is exact.
  int s = 1;
  while ((int64_t{1} << s) < a.period) ++s;
  a.shift = s - 1;
  a.magic = static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + a.period - 1) / a.period);
  a.ldx = d.ldx ? d.ldx : d.D;
  a.eps = d.eps;
  return a;
}

}  // namespace

size_t layernorm_workspace(const ttt_ln_desc& d) {
  return align256(static_cast<size_t>(bwd_slices(d)) * d.groups * 2 * d.D * sizeof(float));
}

hipError_t layernorm_fwd_launch(const ttt_ln_desc& d, const void* x, const void* res, const float* w, const float* b, void* y,
                                void* r, float* mean, float* rstd, hipStream_t s) {
  const Plan p = make_plan(d);
  LnArgs a = make_args(d);
  a.x = x; a.res = res; a.w = w; a.b = b; a.y = y; a.r = r; a.mean = mean; a.rstd = rstd;
  const int unroll = fwd_unroll(d, p);
  a.slices = slices_of(d, p, unroll, fwd_per_cu(d, p));
  a.wpr = p.wpr;
  const dim3 grid(static_cast<uint32_t>(a.slices) * a.G);
  KernelScope scope(TTT_KERNEL_LN_FWD, s);
  if (!p.nit) {
    if (d.dtype == TTT_BF16) ln_fwd_long_kernel<bf16_t><<<grid, kLongThreads, 0, s>>>(a);
    else ln_fwd_long_kernel<float><<<grid, kLongThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  return dispatch<true>(d, p, unroll, res != nullptr, [&](auto e, auto vec, auto tpr, auto nit, auto ur, auto with) {
    ln_fwd_kernel<decltype(e), vec(), tpr(), nit(), ur(), with()><<<grid, p.threads, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t layernorm_bwd_launch(const ttt_ln_desc& d, const void* x, const float* w, const float* mean, const float* rstd,
                                const void* dy, const void* dr, void* dx, float* dw, float* db, void* ws, hipStream_t s) {
  const Plan p = make_plan(d);
  LnArgs a = make_args(d);
  a.x = x; a.w = w; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.dy = dy; a.dr = dr; a.dx = dx;
  a.part = dw || db ? static_cast<float*>(ws) : nullptr;
  const int unroll = bwd_unroll(d, p);
  a.slices = bwd_slices(d);
  a.wpr = p.wpr;
  const dim3 grid(static_cast<uint32_t>(a.slices) * a.G);
  hipError_t st;
  {
    KernelScope scope(TTT_KERNEL_LN_BWD, s);
    if (!p.nit) {
      if (d.dtype == TTT_BF16) ln_bwd_long_kernel<bf16_t><<<grid, kLongThreads, 0, s>>>(a);
      else ln_bwd_long_kernel<float><<<grid, kLongThreads, 0, s>>>(a);
      st = hipGetLastError();
    } else {
      st = dispatch<false>(d, p, unroll, dr != nullptr, [&](auto e, auto vec, auto tpr, auto nit, auto ur, auto with) {
        ln_bwd_kernel<decltype(e), vec(), tpr(), nit(), ur(), with()><<<grid, p.threads, 0, s>>>(a);
        return hipGetLastError();
      });
    }
  }
  if (st != hipSuccess || !a.part) return st;
  const int64_t cols = static_cast<int64_t>(d.groups) * 2 * d.D;
  KernelScope scope(TTT_KERNEL_LN_REDUCE, s);
  const int64_t blocks = std::min<int64_t>((cols + kReduceCols - 1) / kReduceCols, kReduceGrid);
  ln_reduce_kernel<<<static_cast<uint32_t>(blocks), kReduceThreads, 0, s>>>(a.part, a.slices, a.G, a.D, dw, db);
  return hipGetLastError();
}

}  // namespace ttt
