// Layer norm over the rows of [rows, D] on gfx950, forward and backward.
//
//   r = x (+ res, rounded to the tensors' type);  mu, s = 1 / sqrt(var + eps);
//   n = (r - mu) s;  y = n w_g + b_g,  g the row's group (a head's weight, say).
// Backward, with t = w_g dy:
//   dx = s (t - mean(t) - n mean(t n)) (+ dr);  dw_g = sum dy n;  db_g = sum dy.
//
// Both passes are bound by memory: a row is read once into registers, a thread
// holding NIT pieces of VEC elements (16 bytes where the rows allow it).  Narrow
// rows take a part of a wave each, wide rows the whole workgroup, whose size is
// the row's number of pieces.  A workgroup walks over rows of one group, so the
// weights stay in registers, and takes UR rows at a time: their loads are in
// flight together and they share the barriers of a cross-wave sum.  The variance
// is the mean of (r - mu)^2 in a second sum over the registers, exact also where
// the mean is far larger than the deviation.
//
// dw and db: a thread owns its columns, sums them over the workgroup's rows in
// fp32 and writes one partial row; ln_reduce_kernel adds the partial rows in a
// fixed order.

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
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = r[k];
  }
  static __device__ __forceinline__ Raw put(const float (&f)[4]) { return Raw{f[0], f[1], f[2], f[3]}; }
};
template <> struct Piece<bf16_t, 1> {
  using Raw = uint16_t;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) { f[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f32_to_bf16(f[0]); }
};
template <> struct Piece<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void get(const Raw& r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};

// The k-th row of group g.
__device__ __forceinline__ int64_t row_of(const LnArgs& a, int g, int k) {
  if (a.G == 1) return k;
  const int q = k / a.period;
  return (static_cast<int64_t>(q) * a.G + g) * a.period + (k - q * a.period);
}

// The sum of N values over the TPR lanes of a row (TPR <= 64), or over the
// workgroup (TPR == 0, through `lds`, which alternates between two halves so that
// one barrier a call is enough).  Every thread gets the sum; the order is fixed.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds, int& half) {
  constexpr int kLanes = TPR ? TPR : 64;
#pragma unroll
  for (int s = 1; s < kLanes; s <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], s);
  if constexpr (TPR == 0) {
    const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
    if (waves > 1) {
      float* p = lds + half * N * kMaxWaves;
      half ^= 1;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) p[k * kMaxWaves + wave] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float s = 0.0f;
        for (int w = 0; w < waves; ++w) s += p[k * kMaxWaves + w];
        v[k] = s;
      }
    }
  }
}

template <typename E, int VEC, int TPR, int NIT, int UR>
__global__ __launch_bounds__(TPR ? 256 : 1024) void ln_fwd_kernel(LnArgs a) {
  using P = Piece<E, VEC>;
  using Raw = typename P::Raw;
  __shared__ float lds[2 * UR * kMaxWaves];
  int half = 0;
  const int tpr = TPR ? TPR : blockDim.x;
  const int slots = TPR ? 256 / tpr : 1;  // rows side by side
  const int slot = TPR ? threadIdx.x / tpr : 0, tr = TPR ? threadIdx.x % tpr : threadIdx.x;
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  const E* X = static_cast<const E*>(a.x);
  const E* R = static_cast<const E*>(a.res);
  float w[NIT][VEC], b[NIT][VEC];
  bool has[NIT];
#pragma unroll
  for (int i = 0; i < NIT; ++i) {
    const int c = (i * tpr + tr) * VEC;
    has[i] = c < a.D;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = has[i] && a.w ? a.w[static_cast<int64_t>(g) * a.D + c + e] : 1.0f;
      b[i][e] = has[i] && a.b ? a.b[static_cast<int64_t>(g) * a.D + c + e] : 0.0f;
    }
  }
  const float inv = 1.0f / static_cast<float>(a.D);
  for (int64_t k0 = static_cast<int64_t>(slice) * slots * UR; k0 < a.per_group; k0 += static_cast<int64_t>(a.slices) * slots * UR) {
    float f[UR][NIT][VEC], sum[UR];
    int64_t row[UR];
    bool ok[UR];
    Raw xr[UR][NIT], rr[UR][NIT];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int64_t k = k0 + u * slots + slot;
      ok[u] = k < a.per_group;
      row[u] = row_of(a, g, static_cast<int>(ok[u] ? k : 0));
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        const int c = has[i] ? (i * tpr + tr) * VEC : 0;
        xr[u][i] = *reinterpret_cast<const Raw*>(X + row[u] * a.ldx + c);
        if (R) rr[u][i] = *reinterpret_cast<const Raw*>(R + row[u] * a.D + c);
      }
    }
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      sum[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        P::get(xr[u][i], f[u][i]);
        if (R) {
          float q[VEC];
          P::get(rr[u][i], q);
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[u][i][e] += q[e];
          // the stream is normalised as it is kept, so that the backward sees the same rows
          const Raw kept = P::put(f[u][i]);
          P::get(kept, f[u][i]);
          if (ok[u] && has[i]) *reinterpret_cast<Raw*>(static_cast<E*>(a.r) + row[u] * a.D + (i * tpr + tr) * VEC) = kept;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[u] += has[i] ? f[u][i][e] : 0.0f;
      }
    }
    row_sum<TPR, UR>(sum, lds, half);
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
          var[u] += has[i] ? f[u][i][e] * f[u][i][e] : 0.0f;
        }
    }
    row_sum<TPR, UR>(var, lds, half);
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const float s = 1.0f / sqrtf(var[u] * inv + a.eps);
      if (!ok[u]) continue;
      if (tr == 0) {
        if (a.mean) a.mean[row[u]] = mu[u];
        if (a.rstd) a.rstd[row[u]] = s;
      }
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = f[u][i][e] * s * w[i][e] + b[i][e];
        if (has[i]) *reinterpret_cast<Raw*>(static_cast<E*>(a.y) + row[u] * a.D + (i * tpr + tr) * VEC) = P::put(y);
      }
    }
  }
}

template <typename E, int VEC, int TPR, int NIT, int UR>
__global__ __launch_bounds__(TPR ? 256 : 1024) void ln_bwd_kernel(LnArgs a) {
  using P = Piece<E, VEC>;
  using Raw = typename P::Raw;
  __shared__ float lds[4 * UR * kMaxWaves];
  __shared__ float cols[TPR ? 256 * VEC : 1];
  int half = 0;
  const int tpr = TPR ? TPR : blockDim.x;
  const int slots = TPR ? 256 / tpr : 1;
  const int slot = TPR ? threadIdx.x / tpr : 0, tr = TPR ? threadIdx.x % tpr : threadIdx.x;
  const int g = blockIdx.x % a.G, slice = blockIdx.x / a.G;
  const E* X = static_cast<const E*>(a.x);
  const E* DY = static_cast<const E*>(a.dy);
  const E* DR = static_cast<const E*>(a.dr);
  float w[NIT][VEC], dw[NIT][VEC], db[NIT][VEC];
  bool has[NIT];
#pragma unroll
  for (int i = 0; i < NIT; ++i) {
    const int c = (i * tpr + tr) * VEC;
    has[i] = c < a.D;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = has[i] && a.w ? a.w[static_cast<int64_t>(g) * a.D + c + e] : 1.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
  }
  const float inv = 1.0f / static_cast<float>(a.D);
  for (int64_t k0 = static_cast<int64_t>(slice) * slots * UR; k0 < a.per_group; k0 += static_cast<int64_t>(a.slices) * slots * UR) {
    float n[UR][NIT][VEC], t[UR][NIT][VEC], sum[2 * UR], s[UR];
    int64_t row[UR];
    bool ok[UR];
    Raw xr[UR][NIT], yr[UR][NIT], rr[UR][NIT];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const int64_t k = k0 + u * slots + slot;
      ok[u] = k < a.per_group;
      row[u] = row_of(a, g, static_cast<int>(ok[u] ? k : 0));
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        const int c = has[i] ? (i * tpr + tr) * VEC : 0;
        xr[u][i] = *reinterpret_cast<const Raw*>(X + row[u] * a.ldx + c);
        yr[u][i] = *reinterpret_cast<const Raw*>(DY + row[u] * a.D + c);
        if (DR) rr[u][i] = *reinterpret_cast<const Raw*>(DR + row[u] * a.D + c);
      }
    }
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      const float mu = a.mean[row[u]];
      s[u] = a.rstd[row[u]];
      sum[2 * u] = sum[2 * u + 1] = 0.0f;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        P::get(xr[u][i], n[u][i]);
        P::get(yr[u][i], t[u][i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float dy = t[u][i][e];
          n[u][i][e] = (n[u][i][e] - mu) * s[u];
          if (ok[u]) {
            dw[i][e] += dy * n[u][i][e];
            db[i][e] += dy;
          }
          t[u][i][e] = w[i][e] * dy;
          sum[2 * u] += has[i] ? t[u][i][e] : 0.0f;
          sum[2 * u + 1] += has[i] ? t[u][i][e] * n[u][i][e] : 0.0f;
        }
      }
    }
    row_sum<TPR, 2 * UR>(sum, lds, half);
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      if (!ok[u]) continue;
      const float m1 = sum[2 * u] * inv, m2 = sum[2 * u + 1] * inv;
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        float d[VEC], q[VEC];
        if (DR) P::get(rr[u][i], q);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          d[e] = s[u] * (t[u][i][e] - m1 - n[u][i][e] * m2);
          if (DR) d[e] += q[e];
        }
        if (has[i]) *reinterpret_cast<Raw*>(static_cast<E*>(a.dx) + row[u] * a.ldx + (i * tpr + tr) * VEC) = P::put(d);
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + (static_cast<int64_t>(slice) * a.G + g) * 2 * a.D;
  if constexpr (TPR) {
    // the rows side by side: their sums meet in LDS, the first row's threads add them up
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int i = 0; i < NIT; ++i) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) cols[threadIdx.x * VEC + e] = which ? db[i][e] : dw[i][e];
        __syncthreads();
        if (slot == 0 && has[i]) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float v = 0.0f;
            for (int q = 0; q < slots; ++q) v += cols[(q * tpr + tr) * VEC + e];
            out[which * a.D + (i * tpr + tr) * VEC + e] = v;
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NIT; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (has[i]) {
          out[(i * tpr + tr) * VEC + e] = dw[i][e];
          out[a.D + (i * tpr + tr) * VEC + e] = db[i][e];
        }
  }
}

// Rows that no workgroup holds in registers: every sum walks over the row again.
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
    row_sum<0, 1>(sum, lds, half);
    const float mu = sum[0] * inv;
    const E* src = q ? r : x;  // each thread reads the columns that it wrote
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float f = Elem<E>::ld(src, c) - mu;
      var[0] += f * f;
    }
    row_sum<0, 1>(var, lds, half);
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
    row_sum<0, 2>(sum, lds, half);
    const float m1 = sum[0] * inv, m2 = sum[1] * inv;
    for (int c = threadIdx.x; c < a.D; c += kLongThreads) {
      const float n = (Elem<E>::ld(x, c) - mu) * s, t = Elem<E>::ld(dy, c) * (w ? w[c] : 1.0f);
      Elem<E>::st(dx, c, s * (t - m1 - n * m2) + (dr ? Elem<E>::ld(dr, c) : 0.0f));
    }
  }
}

// dw[g][c], db[g][c] = the sum of their `slices` partial rows: 64 columns a
// workgroup, its waves each add a part of the rows.
constexpr int kReduceWaves = 16;

__global__ __launch_bounds__(kReduceWaves * 64) void ln_reduce_kernel(const float* __restrict__ part, int slices, int G, int D,
                                                                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sums[kReduceWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t cols = static_cast<int64_t>(G) * 2 * D;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float v = 0.0f;
  if (c < cols)
    for (int s = wave; s < slices; s += kReduceWaves) v += part[s * cols + c];
  sums[wave][lane] = v;
  __syncthreads();
  if (wave != 0 || c >= cols) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kReduceWaves; ++w) v += sums[w][lane];
  const int64_t g = c / (2 * D), q = c - g * 2 * D;
  float* to = q < D ? dw : db;
  if (to) to[g * D + (q < D ? q : q - D)] = v;
}

// ---- host ----

// How a row is laid over threads.
struct Plan {
  int vec;      // elements of a piece
  int tpr;      // lanes of a row (8 .. 64), or 0: the workgroup
  int nit;      // pieces of a thread; 0: the long kernels
  int threads;  // of a workgroup
  int slots;    // rows side by side
};

Plan make_plan(const ttt_ln_desc& d) {
  const int wide = d.dtype == TTT_BF16 ? 8 : 4;
  const int64_t ldx = d.ldx ? d.ldx : d.D;
  Plan p{};
  p.vec = d.D % wide == 0 && ldx % wide == 0 ? wide : 1;
  const int pieces = (d.D + p.vec - 1) / p.vec;
  if (pieces <= 64) {
    p.tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    p.nit = 1;
    p.threads = 256;
    p.slots = 256 / p.tpr;
    return p;
  }
  p.slots = 1;
  p.nit = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : pieces <= 4096 ? 4 : 0;
  p.threads = p.nit ? ((pieces + p.nit - 1) / p.nit + 63) / 64 * 64 : kLongThreads;
  return p;
}

// Workgroups of each group: enough for every CU to hold several, and no more than
// there are rows for (`unroll` of them a step).
int slices_of(const ttt_ln_desc& d, const Plan& p, int unroll, int per_cu) {
  const int per_group = static_cast<int>(d.rows / d.groups);
  const int64_t steps = (static_cast<int64_t>(per_group) + p.slots * unroll - 1) / (p.slots * unroll);
  const int64_t want = (256 * per_cu + d.groups - 1) / d.groups;
  const int64_t n = steps < want ? steps : want;
  return static_cast<int>(n > 0 ? n : 1);
}

constexpr int kFwdPerCu = 8, kBwdPerCu = 2;
// Rows a workgroup takes at once; few rows go to as many workgroups as there are.
int unroll_of(const ttt_ln_desc& d, const Plan& p) {
  if (p.nit > 1) return 1;
  return d.rows >= 4096 * p.slots ? 4 : 1;
}

int bwd_slices(const ttt_ln_desc& d) {
  const Plan p = make_plan(d);
  return slices_of(d, p, p.nit ? unroll_of(d, p) : 1, kBwdPerCu);
}

template <typename F> hipError_t dispatch(const ttt_ln_desc& d, const Plan& p, int unroll, F&& f) {
  auto with_rows = [&](auto e, auto vec, auto tpr, auto nit) {
    if constexpr (nit() == 1) {
      if (unroll == 4) return f(e, vec, tpr, nit, std::integral_constant<int, 4>{});
    }
    return f(e, vec, tpr, nit, std::integral_constant<int, 1>{});
  };
  auto with_plan = [&](auto e, auto vec) {
    std::integral_constant<int, 1> one;
    switch (p.tpr) {
      case 8: return with_rows(e, vec, std::integral_constant<int, 8>{}, one);
      case 16: return with_rows(e, vec, std::integral_constant<int, 16>{}, one);
      case 32: return with_rows(e, vec, std::integral_constant<int, 32>{}, one);
      case 64: return with_rows(e, vec, std::integral_constant<int, 64>{}, one);
    }
    std::integral_constant<int, 0> group;
    if (p.nit == 1) return with_rows(e, vec, group, one);
    if (p.nit == 2) return with_rows(e, vec, group, std::integral_constant<int, 2>{});
    return with_rows(e, vec, group, std::integral_constant<int, 4>{});
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
  const int unroll = p.nit ? unroll_of(d, p) : 1;
  a.slices = slices_of(d, p, unroll, kFwdPerCu);
  const dim3 grid(static_cast<uint32_t>(a.slices) * a.G);
  KernelScope scope(TTT_KERNEL_LN_FWD, s);
  if (!p.nit) {
    if (d.dtype == TTT_BF16) ln_fwd_long_kernel<bf16_t><<<grid, kLongThreads, 0, s>>>(a);
    else ln_fwd_long_kernel<float><<<grid, kLongThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  return dispatch(d, p, unroll, [&](auto e, auto vec, auto tpr, auto nit, auto ur) {
    ln_fwd_kernel<decltype(e), vec(), tpr(), nit(), ur()><<<grid, p.threads, 0, s>>>(a);
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
  const int unroll = p.nit ? unroll_of(d, p) : 1;
  a.slices = bwd_slices(d);
  const dim3 grid(static_cast<uint32_t>(a.slices) * a.G);
  hipError_t st;
  {
    KernelScope scope(TTT_KERNEL_LN_BWD, s);
    if (!p.nit) {
      if (d.dtype == TTT_BF16) ln_bwd_long_kernel<bf16_t><<<grid, kLongThreads, 0, s>>>(a);
      else ln_bwd_long_kernel<float><<<grid, kLongThreads, 0, s>>>(a);
      st = hipGetLastError();
    } else {
      st = dispatch(d, p, unroll, [&](auto e, auto vec, auto tpr, auto nit, auto ur) {
        ln_bwd_kernel<decltype(e), vec(), tpr(), nit(), ur()><<<grid, p.threads, 0, s>>>(a);
        return hipGetLastError();
      });
    }
  }
  if (st != hipSuccess || !a.part) return st;
  const int64_t cols = static_cast<int64_t>(d.groups) * 2 * d.D;
  KernelScope scope(TTT_KERNEL_LN_REDUCE, s);
  ln_reduce_kernel<<<static_cast<uint32_t>((cols + 63) / 64), kReduceWaves * 64, 0, s>>>(a.part, a.slices, a.G, a.D, dw, db);
  return hipGetLastError();
}

}  // namespace ttt
