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
// packed case with a start every T tokens).  A tile is kWaves LW tokens x 64
// V channels; a wave holds LW tokens of it in registers, V channels a lane, and the
// waves' maps meet in LDS.  The backward keeps its inputs packed as they were loaded
// and forms a_t again in each of its three walks: that costs arithmetic, of which
// there is room, and saves registers, of which there is none.
//
// Tiles meet through memory, in one pass over the data: a tile publishes its map
// as soon as it has it, then reads the maps of the tiles before it (after it, in
// the backward), folds them in their order and writes its outputs from the value
// that enters it.  A sequence start inside a tile makes its map independent of
// what enters, so a tile reads back to the tile where the sequence of its first
// token starts, and no further; over long ways it reads the maps of whole groups
// of kGroup tiles, which each group's last tile publishes.
// - A map is one 8-byte word (A, B) a channel, stored and loaded whole at agent
//   scope, so a word that is not all ones is complete: no fence, no flag.
// - Every wait ends: a workgroup takes its place on the token axis from a counter
//   (one a channel block) when it starts to run, so the tiles that it waits for
//   are held by workgroups that run already, and these publish before they wait.
//   A group's map depends on its tiles' maps alone.  Should a caller break the
//   rule of one workspace a call all the same, the wait gives up after kPolls
//   looks and the outputs are NaN.
// - The fold's order is fixed by the tiles' places, so results repeat to the bit.
//
// Starts are the same for every channel, so all control flow on them is
// wave-uniform.  The state of another sequence is never multiplied in (not even
// by zero): a NaN or an infinity stays in its sequence.

#include <cstdint>
#include <type_traits>

#include "ttt_device.h"
#include "ttt_internal.h"

namespace ttt {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kBwdLW = 16;           // tokens a wave holds in the backward
constexpr int kRun = kWaves * kBwdLW;  // tokens between two states in the saved context
constexpr int kGroup = 32;           // tiles of a group
constexpr int kCounterStride = 32;   // ints between two channel blocks' counters: a cache line each
constexpr int kPolls = 1 << 20;      // of a wave, together; a look takes about a microsecond

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
  float* ckpt;  // [runs][Dp]: the state that enters each run of kRun tokens
  uint64_t* maps;    // [nt][Dp]: each tile's map, all ones until it is there
  uint64_t* groups;  // [ng][Dp]: each whole group's
  int* counters;     // [ncb]: tiles taken
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
  static constexpr Raw kInf = __builtin_inff();
  static __device__ __forceinline__ void get(Raw r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f[0]; }
};
template <> struct Io<bf16_t, 1> {
  using Raw = uint16_t;
  static constexpr Raw kInf = 0x7f80;
  static __device__ __forceinline__ void get(Raw r, float (&f)[1]) { f[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ Raw put(const float (&f)[1]) { return f32_to_bf16(f[0]); }
};
template <> struct Io<bf16_t, 2> {
  using Raw = uint32_t;
  static constexpr Raw kInf = 0x7f807f80u;
  static __device__ __forceinline__ void get(Raw r, float (&f)[2]) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw put(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
};

// A value that is the same in every lane, kept as such.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const char*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Up to LW rows of a tensor from row t on, as a buffer resource over just them: a
// load past them reads zero and a store past them does nothing, so neither the
// last tile's rows nor the last block's lanes need a branch.
// A range is at most 2^30 bytes: kNowhere, as a lane's offset, stays behind it for
// every row, and so does kNoRow in place of a row's, added to either kind of lane.
constexpr uint32_t kNowhere = 0x40000000u, kNoRow = 0x80000000u;
template <typename Raw, int LW> struct Rows {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t stride;  // bytes from row to row, at most 2^30 / LW
  __device__ __forceinline__ Rows(const void* base, int64_t ld, int D, int elem, int t, int n) {
    const int rows = min(max(n - t, 0), LW);
    const uint32_t bytes = rows > 0 ? static_cast<uint32_t>(rows - 1) * static_cast<uint32_t>(ld * elem) + D * elem : 0;
    const char* p = uniform(static_cast<const char*>(base) + (rows > 0 ? t * ld * elem : 0));
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, uniform(static_cast<int>(bytes)), 0x00020000);
    stride = uniform(static_cast<int>(ld * elem));
  }
  __device__ __forceinline__ Raw load(int j, uint32_t off) const {
    if constexpr (sizeof(Raw) == 2) return __builtin_amdgcn_raw_buffer_load_b16(rs, static_cast<int>(off + j * stride), 0, 0);
    else return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(off + j * stride), 0, 0));
  }
  __device__ __forceinline__ void store(int j, uint32_t off, bool ok, Raw v) const {  // ok: the same for the wave
    const int at = static_cast<int>(off + (ok ? j * stride : kNoRow));
    if constexpr (sizeof(Raw) == 2) __builtin_amdgcn_raw_buffer_store_b16(v, rs, at, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rs, at, 0, 0);
  }
};

template <typename Raw> __device__ __forceinline__ Raw load_at(const void* base, int64_t row_bytes, uint32_t off) {
  return *reinterpret_cast<const Raw*>(static_cast<const char*>(base) + row_bytes + off);
}
template <typename Raw> __device__ __forceinline__ void store_at(void* base, int64_t row_bytes, uint32_t off, Raw v) {
  *reinterpret_cast<Raw*>(static_cast<char*>(base) + row_bytes + off) = v;
}

// The same value, of which the compiler knows nothing: what was formed from it
// before is formed again, not kept in registers.
template <typename Raw> __device__ __forceinline__ Raw afresh(Raw r) {
  if constexpr (sizeof(Raw) == 2) {
    uint32_t q = r;
    asm volatile("" : "+v"(q));
    r = static_cast<Raw>(q);
  } else {
    asm volatile("" : "+v"(r));
  }
  return r;
}

// Bit j of a mask that is the same for the wave, tested where it is asked: the
// compiler would keep the results of all tests in scalar registers otherwise.
__device__ __forceinline__ bool bit(uint32_t mask, int j) {
  asm volatile("" : "+s"(mask));
  return mask >> j & 1;
}

// Keeps the compiler from forming the coefficients of many tokens ahead, which
// would hold them all in registers; the other waves hide the latency instead.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

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
template <int LW> struct Meta {
  static constexpr int kTile = kWaves * LW;
  int start[kTile], end[kTile];
  int lo, hi, first, last;
};
// The same for one wave's tokens: bits of those that belong to a sequence, start
// one, end one.  inside: the whole tile lies inside one sequence, without its start
// or its end.  first, last: as in Meta, or the tile's own first and last token
// where it has none of a sequence.
struct Bits {
  bool inside;
  uint32_t ok, start, end;
  int first, last;
};
template <int LW> constexpr uint32_t kAll = static_cast<uint32_t>((uint64_t{1} << LW) - 1);

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

template <int LW> __device__ __forceinline__ Bits tile_meta(const RecArgs& a, int t0, Meta<LW>& m) {
  constexpr int kTile = Meta<LW>::kTile;
  const int tid = threadIdx.x;
  const int tl = t0 + kTile - 1;
  bool one = false;  // the first and the last token are of the same sequence
  if (!a.starts) {
    if (tl < a.n) {
      const int from = t0 - t0 % a.T;
      // inside one sequence, and neither its start nor its end
      if (from < t0 && from + a.T - 1 > tl) return Bits{true, kAll<LW>, 0, 0, from, from + a.T - 1};
    }
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
    one = uniform(sl) == uniform(s0);
    if (tid == 0) {
      m.lo = max(t0, a.starts[0]);
      m.hi = min(min(t0 + kTile, a.n), a.starts[a.B]);
      m.first = min(max(a.starts[s0], 0), t0);
      m.last = sl < 0 || sl >= a.B ? tl : min(max(a.starts[sl + 1], tl + 1) - 1, max(a.n - 1, tl));
    }
  }
  __syncthreads();
  const int lo = uniform(m.lo), hi = uniform(m.hi), first = uniform(m.first), last = uniform(m.last);
  if (one && lo <= t0 && hi > tl && first < t0 && last > tl) return Bits{true, kAll<LW>, 0, 0, first, last};
  const int lane = tid & 63, at = (tid >> 6) * LW + lane % LW, t = t0 + at;
  const bool ok = lane < LW && t >= lo && t < hi;
  return Bits{false, static_cast<uint32_t>(__ballot(ok)), static_cast<uint32_t>(__ballot(ok && m.start[at] >= 0)),
              static_cast<uint32_t>(__ballot(ok && m.end[at] >= 0)), lo < hi ? first : t0, lo < hi ? last : tl};
}

// Sequences without a token: the state passes through (dst = src, or zero).
// Tile i of the grid takes its share of the sequences, a wave one at a time.
template <int V>
__device__ __forceinline__ void pass_empty(const RecArgs& a, int i, int c, bool in, const float* src, float* dst) {
  if (!dst) return;
  if (!a.starts && a.T > 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s1 = static_cast<int>(static_cast<int64_t>(a.B) * (i + 1) / a.nt);
  for (int s = static_cast<int>(static_cast<int64_t>(a.B) * i / a.nt) + wave; s < s1; s += kWaves) {
    if (a.starts && a.starts[s + 1] > a.starts[s]) continue;
    const int64_t at = static_cast<int64_t>(s) * a.D + c;
    if (in) {
#pragma unroll
      for (int v = 0; v < V; ++v) dst[at + v] = src ? src[at + v] : 0.0f;
    }
  }
}

// The map of a run of tokens as one word.  A B of all ones (a NaN that no
// arithmetic makes) would read as pending and becomes another NaN.
__device__ __forceinline__ void publish(uint64_t* p, float A, float B) {
  const uint32_t hi = __float_as_uint(B) == 0xffffffffu ? 0x7fc00000u : __float_as_uint(B);
  __hip_atomic_store(p, static_cast<uint64_t>(hi) << 32 | __float_as_uint(A), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Folds `count` maps onto (A, B), count <= N: all are loaded at once, and again
// while one of them is pending (a pending word reads as NaN).  addr(k): the first
// of the lane's V words.
template <int V, int N, typename Addr>
__device__ __forceinline__ void fold_some(int count, Addr addr, bool reset_first, int& polls, float (&A)[V], float (&B)[V]) {
  uint64_t q[N][V];
  while (true) {
    bool pending = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t* p = addr(k < count ? k : 0);
#pragma unroll
      for (int v = 0; v < V; ++v) q[k][v] = __hip_atomic_load(p + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) pending |= static_cast<uint32_t>(q[k][v] >> 32) == 0xffffffffu;
    if (__ballot(pending) == 0 || --polls <= 0) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k < count) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float qa = __uint_as_float(static_cast<uint32_t>(q[k][v])), qb = __uint_as_float(static_cast<uint32_t>(q[k][v] >> 32));
        const bool reset = k == 0 && reset_first;
        B[v] = reset ? qb : qa * B[v] + qb;
        A[v] = reset ? 0.0f : qa * A[v];
      }
    }
  }
}

// The tiles whose maps enter tile i, from tile `far` on, in their order: far's own
// group up to its border as tiles, then whole groups, then the tiles of i's group.
// dir = 1: tiles before i; -1: behind it.  Groups are counted in the direction, so
// that in the backward a "group" is the same set of tiles read from the end.
struct Way {
  int far, n1, group, n2, near, n3, dir;
  __device__ __forceinline__ Way(int i, int far_, int dir_) : far(far_), dir(dir_) {
    const int gi = i / kGroup, gf = far / kGroup;
    if (gi == gf) {
      n1 = n2 = 0;
      group = 0;
      near = far;
      n3 = dir > 0 ? i - far : far - i;
    } else if (dir > 0) {
      n1 = (gf + 1) * kGroup - far;
      group = gf + 1;
      n2 = gi - gf - 1;
      near = gi * kGroup;
      n3 = i - near;
    } else {
      n1 = far - gf * kGroup + 1;
      group = gf - 1;
      n2 = gf - gi - 1;
      near = (gi + 1) * kGroup - 1;
      n3 = near - i;
    }
  }
  __device__ __forceinline__ int count() const { return n1 + n2 + n3; }
  __device__ __forceinline__ const uint64_t* at(const RecArgs& a, int k, int c) const {
    const bool tile1 = k < n1, grp = !tile1 && k < n1 + n2;
    const int row = tile1 ? far + dir * k : grp ? group + dir * (k - n1) : near + dir * (k - n1 - n2);
    return (grp ? a.groups : a.maps) + static_cast<int64_t>(row) * a.Dp + c;
  }
};

// The value that enters tile i.  The farthest tile's map has a reset in it, so only
// its B counts.  Each wave folds a part, the parts meet in `look`.
template <int V>
__device__ __forceinline__ void fold_way(const RecArgs& a, const Way& way, int c, float (&look)[kWaves][64][2 * V], float (&h)[V]) {
  constexpr int N = 4;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int count = way.count();
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = 0.0f;
  if (count <= 0) return;  // the same for the whole workgroup
  const int k0 = static_cast<int>(static_cast<int64_t>(count) * wave / kWaves);
  const int k1 = static_cast<int>(static_cast<int64_t>(count) * (wave + 1) / kWaves);
  int polls = kPolls;
  float A[V], B[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
  for (int k = k0; k < k1; k += N)
    fold_some<V, N>(min(N, k1 - k), [&](int j) { return way.at(a, k + j, c); }, k == 0, polls, A, B);
#pragma unroll
  for (int v = 0; v < V; ++v) look[wave][lane][2 * v] = A[v], look[wave][lane][2 * v + 1] = B[v];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = look[w][lane][2 * v] * h[v] + look[w][lane][2 * v + 1];
}

// Tile i's map (A, B) goes out; the last tile of a group (in direction dir) then
// publishes the group's.  Wave 0 holds the map.
template <int V>
__device__ __forceinline__ void publish_tile(const RecArgs& a, int i, int dir, int c, float (&look)[kWaves][64][2 * V],
                                             const float (&A)[V], const float (&B)[V]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) publish(a.maps + static_cast<int64_t>(i) * a.Dp + c + v, A[v], B[v]);
  }
  const int g = i / kGroup, from = dir > 0 ? g * kGroup : g * kGroup + kGroup - 1;
  // only a whole group has a map, and only its last tile publishes it
  if (i != (dir > 0 ? g * kGroup + kGroup - 1 : g * kGroup) || (g + 1) * kGroup > a.nt) return;
  constexpr int N = kGroup / kWaves;
  float GA[V], GB[V];
#pragma unroll
  for (int v = 0; v < V; ++v) GA[v] = 1.0f, GB[v] = 0.0f;
  const int count = wave == kWaves - 1 ? N - 1 : N;  // all but tile i itself
  int polls = kPolls;
  fold_some<V, N>(count, [&](int j) { return a.maps + static_cast<int64_t>(from + dir * (wave * N + j)) * a.Dp + c; }, false, polls,
                  GA, GB);
#pragma unroll
  for (int v = 0; v < V; ++v) look[wave][lane][2 * v] = GA[v], look[wave][lane][2 * v + 1] = GB[v];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float qa = look[w][lane][2 * v], qb = look[w][lane][2 * v + 1];
        GB[v] = qa * GB[v] + qb;
        GA[v] = qa * GA[v];
      }
#pragma unroll
    for (int v = 0; v < V; ++v) publish(a.groups + static_cast<int64_t>(g) * a.Dp + c + v, A[v] * GA[v], A[v] * GB[v] + B[v]);
  }
  __syncthreads();  // `look` is free again
}

// The tile that this workgroup works on: the next one of its channel block (place
// 0 is the first in the direction of the run).
__device__ __forceinline__ int take_tile(const RecArgs& a, int cb, int dir) {
  __shared__ int place;
  if (threadIdx.x == 0)
    place = __hip_atomic_fetch_add(a.counters + cb * kCounterStride, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const int p = min(max(__builtin_amdgcn_readfirstlane(place), 0), a.nt - 1);
  return dir > 0 ? p : a.nt - 1 - p;
}

// Every map pending, every counter at zero.  A kernel, not a memset: a graph may hold
// it.  1 to 6 us.
__global__ __launch_bounds__(256) void rec_clear_kernel(uint4* __restrict__ maps, int64_t n, int* __restrict__ counters, int nc) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) maps[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  if (i < nc) counters[i] = 0;
}

// The forward.  Reads x and z and writes o once, in one pass.  Bound by memory on long
// problems: 131072 x 2048 bf16 380 to 390 us, 4.1 to 4.2 TB/s (a copy 4.8).  The same
// kernel without any exchange of maps takes 326: a tile of 192 KB reads 53 KB of them on
// average, from L2 (what comes from beyond it is 1.01 times x and z).  Two bf16 channels
// and 32 tokens a wave take 165 registers, so a CU has one workgroup, whose loads, walks,
// map, look back and stores follow one another: 37 packed prompts, 30011 x 2560 (2360
// tiles, 9.2 rounds), 134 us, 3.4 TB/s, and 110 without the exchange.  16 tokens a wave
// (110 registers, two workgroups) are bound by the same latencies: 4 x 4096 x 2048 bf16
// 61 us, 3.3 TB/s, 45 without the exchange.  f32 has room for four workgroups: 19
// sequences of 9001 x 1001 (1.1 rounds) 41 us, 2.6 TB/s; their rows of 4004 bytes share
// cache lines between channel blocks, and 1.5 times x and z come from beyond the L2.
// LINKED: there is more than one tile.
template <typename E, int V, int GATE, int IN, int LW, bool LINKED>
__global__ __launch_bounds__(kThreads, LW == 32 ? 2 : 4) void rec_fwd_kernel(RecArgs a) {
  using IO = Io<E, V>;
  using Raw = typename IO::Raw;
  __shared__ Meta<LW> m;
  __shared__ __attribute__((aligned(16))) float part[kWaves][64][2 * V];
  __shared__ __attribute__((aligned(16))) float look[kWaves][64][2 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb = blockIdx.x % a.ncb;
  const int i = LINKED ? take_tile(a, cb, 1) : 0;
  const int c = (cb * 64 + lane) * V;
  const bool in = c < a.D;
  const uint32_t cl = in ? c : 0;
  const uint32_t off = in ? c * sizeof(E) : kNowhere;
  const int t0 = i * kWaves * LW, tw = t0 + wave * LW;

  Raw xr[LW], gr[LW];
  const Rows<Raw, LW> xs(a.x, a.ldx, a.D, sizeof(E), tw, a.n), gs(a.g, a.ldg, a.D, sizeof(E), tw, a.n);
#pragma unroll
  for (int j = 0; j < LW; ++j) gr[j] = gs.load(j, off), xr[j] = xs.load(j, off);
  const Bits bits = tile_meta<LW>(a, t0, m);
  const uint32_t okm = uniform(bits.ok), sm = uniform(bits.start), em = uniform(bits.end);
  if (okm != kAll<LW>) {
    // a token of no sequence: a = 1 and u = 0 leave what passes over it as it is
#pragma unroll
    for (int j = 0; j < LW; ++j)
      if (!(okm >> j & 1)) xr[j] = Raw(0), gr[j] = GATE == TTT_GATE_SIGMOID ? IO::kInf : Raw(0);
  }
  float f[LW][V], u[LW][V];
#pragma unroll
  for (int j = 0; j < LW; ++j) {
    float x[V], z[V];
    IO::get(xr[j], x);
    IO::get(gr[j], z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f[j][v] = gate_a<GATE>(z[v]);
      u[j][v] = IN == TTT_REC_PLAIN ? x[v] : gate_rest<GATE>(z[v], f[j][v]) * x[v];
    }
  }
  float A[V], h[V];
  auto initial = [&](int j) {  // h0 of the sequence that starts at the wave's token j
    const int s = uniform(m.start[wave * LW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = a.h0 ? a.h0[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };

  // The map of the wave's tokens.  Both walks have a form without tests for the waves
  // that lie inside one sequence; only the short walks are there twice, since a kernel
  // with two whole bodies took 10% longer in either.
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.0f, h[v] = 0.0f;
  if (sm == 0) {
#pragma unroll
    for (int j = 0; j < LW; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = f[j][v] * h[v] + u[j][v];
        A[v] *= f[j][v];
      }
  } else {
    // what enters counts no longer behind a start: the sign of A says so to the readers of `part`
#pragma unroll
    for (int j = 0; j < LW; ++j) {
      if (sm >> j & 1) initial(j);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = f[j][v] * h[v] + u[j][v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = -1.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) part[wave][lane][2 * v] = A[v], part[wave][lane][2 * v + 1] = h[v];
  __syncthreads();

  // fold the maps of waves 0 .. upto - 1 onto h; A: the product, dropped at a start
  auto fold_waves = [&](int upto) {
    for (int w = 0; w < upto; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float pa = part[w][lane][2 * v], pb = part[w][lane][2 * v + 1];
        const bool reset = pa < 0.0f;
        h[v] = reset ? pb : pa * h[v] + pb;
        A[v] = reset ? 0.0f : pa * A[v];
      }
    }
  };
  if constexpr (LINKED) {
    if (wave == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) A[v] = 1.0f, h[v] = 0.0f;
      fold_waves(kWaves);
    }
    publish_tile<V>(a, i, 1, c, look, A, h);
    fold_way<V>(a, Way(i, uniform(bits.first) / (kWaves * LW), 1), c, look, h);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.0f;
  }
  fold_waves(wave);
  if (a.ckpt && (wave * LW) % kRun == 0 && tw < a.n) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.ckpt[static_cast<int64_t>(tw / kRun) * a.Dp + c + v] = h[v];
  }
  const Rows<Raw, LW> os(a.o, a.D, a.D, sizeof(E), tw, a.n);
  if (okm == kAll<LW> && (sm | em) == 0) {
#pragma unroll
    for (int j = 0; j < LW; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = f[j][v] * h[v] + u[j][v];
      os.store(j, off, true, IO::put(h));
    }
  } else {
#pragma unroll
    for (int j = 0; j < LW; ++j) {
      if (sm >> j & 1) initial(j);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = f[j][v] * h[v] + u[j][v];
      os.store(j, off, okm >> j & 1, IO::put(h));
      if (in && a.h_final && (em >> j & 1)) {
        const int s = uniform(m.end[wave * LW + j]);
#pragma unroll
        for (int v = 0; v < V; ++v) a.h_final[static_cast<int64_t>(s) * a.D + c + v] = h[v];
      }
    }
  }
  pass_empty<V>(a, i, c, in, a.h0, a.h_final);
}

// The backward: the same tiles, e running from the end.  The tile's states are
// formed again from the state that entered it (ckpt) and the waves' forward maps, so
// h is neither kept nor read.  Bound by memory and by the three walks' arithmetic
// (a_t formed in each): 4 x 4096 x 2048 bf16 85 us for 336 MB, 3.9 TB/s; 9001 x 1001 f32
// (91 registers, two workgroups a CU, 2.2 rounds) 56 us for 180 MB, 3.2 TB/s.
template <typename E, int V, int GATE, int IN, int LW, bool LINKED>
__global__ __launch_bounds__(kThreads, 4) void rec_bwd_kernel(RecArgs a) {
  static_assert(kWaves * LW == kRun, "a tile starts where the forward saved a state");
  using IO = Io<E, V>;
  using Raw = typename IO::Raw;
  __shared__ Meta<LW> m;
  __shared__ __attribute__((aligned(16))) float part[kWaves][64][2 * V];   // the waves' maps of h
  __shared__ __attribute__((aligned(16))) float rpart[kWaves][64][2 * V];  // and of e, from the end
  __shared__ __attribute__((aligned(16))) float look[kWaves][64][2 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb = blockIdx.x % a.ncb;
  const int i = LINKED ? take_tile(a, cb, -1) : 0;
  const int c = (cb * 64 + lane) * V;
  const bool in = c < a.D;
  const uint32_t cl = in ? c : 0;
  const uint32_t off = in ? c * sizeof(E) : kNowhere;
  const int t0 = i * kWaves * LW, tw = t0 + wave * LW;

  Raw xr[LW], gr[LW], dr[LW];
  const Rows<Raw, LW> xs(a.x, a.ldx, a.D, sizeof(E), tw, a.n), gs(a.g, a.ldg, a.D, sizeof(E), tw, a.n);
  const Rows<Raw, LW> ds(a.d_o, a.D, a.D, sizeof(E), tw, a.n);
#pragma unroll
  for (int j = 0; j < LW; ++j) gr[j] = gs.load(j, off), xr[j] = xs.load(j, off), dr[j] = ds.load(j, off);
  const Bits bits = tile_meta<LW>(a, t0, m);
  const uint32_t okm = uniform(bits.ok), sm = uniform(bits.start), em = uniform(bits.end);
  if (okm != kAll<LW>) {
#pragma unroll
    for (int j = 0; j < LW; ++j)
      if (!(okm >> j & 1)) xr[j] = dr[j] = Raw(0), gr[j] = GATE == TTT_GATE_SIGMOID ? IO::kInf : Raw(0);
  }
  const bool inner = okm == kAll<LW> && (sm | em) == 0;  // the wave lies inside one sequence
  float h[V], e[V], P[V];
  auto coefficients = [&](int j, float (&f)[V], float (&rest)[V]) {
    float z[V];
    IO::get(afresh(gr[j]), z);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f[v] = gate_a<GATE>(z[v]);
      rest[v] = gate_rest<GATE>(z[v], f[v]);
    }
  };
  auto initial = [&](int j) {
    const int s = uniform(m.start[wave * LW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = a.h0 ? a.h0[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };
  auto final_grad = [&](int j, float (&q)[V]) {
    const int s = uniform(m.end[wave * LW + j]);
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = a.d_hfinal ? a.d_hfinal[static_cast<int64_t>(s) * a.D + cl + v] : 0.0f;
  };

  // Both maps of the wave's tokens in one walk: with P_j = a_0 ... a_j, h <- a h + u
  // as in the forward, and e in front of the tokens is sum_j P_j do_j + P_last e
  // behind them.  The first end cuts that sum: behind its token only d_hfinal adds.
  float cut[V];
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 1.0f, h[v] = e[v] = cut[v] = 0.0f;
  auto both_maps = [&](auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
    for (int j = 0; j < LW; ++j) {
      in_order();
      if (EDGE && bit(sm, j)) initial(j);
      float f[V], rest[V], x[V], d[V];
      coefficients(j, f, rest);
      IO::get(afresh(xr[j]), x);
      IO::get(afresh(dr[j]), d);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = f[v] * h[v] + (IN == TTT_REC_PLAIN ? x[v] : rest[v] * x[v]);
        P[v] *= f[v];
        e[v] += P[v] * d[v];
      }
      if (EDGE && bit(em, j) && (em & ((1u << j) - 1)) == 0) {
        final_grad(j, cut);
#pragma unroll
        for (int v = 0; v < V; ++v) cut[v] = e[v] + P[v] * cut[v];
      }
    }
  };
  if (inner) both_maps(std::false_type{});
  else both_maps(std::true_type{});
#pragma unroll
  for (int v = 0; v < V; ++v) {
    part[wave][lane][2 * v] = sm ? -1.0f : P[v];
    part[wave][lane][2 * v + 1] = h[v];
    rpart[wave][lane][2 * v] = em ? -1.0f : P[v];
    rpart[wave][lane][2 * v + 1] = em ? cut[v] : e[v];
  }
  __syncthreads();

  // fold the maps of e of waves kWaves - 1 .. from onto e; P: the product
  auto fold_back = [&](int from) {
    for (int w = kWaves - 1; w >= from; --w) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float pa = rpart[w][lane][2 * v], pb = rpart[w][lane][2 * v + 1];
        const bool reset = pa < 0.0f;
        e[v] = reset ? pb : pa * e[v] + pb;
        P[v] = reset ? 0.0f : pa * P[v];
      }
    }
  };
  if constexpr (LINKED) {
    if (wave == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) P[v] = 1.0f, e[v] = 0.0f;
      fold_back(0);
    }
    publish_tile<V>(a, i, -1, c, look, P, e);
  }
  // h_{t-1} of every token, kept as w_t = a'_t (h_{t-1} - (0 or x_t))
  float wv[LW][V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = a.ckpt[static_cast<int64_t>(i) * a.Dp + c + v];
  for (int w = 0; w < wave; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float pa = part[w][lane][2 * v], pb = part[w][lane][2 * v + 1];
      h[v] = pa < 0.0f ? pb : pa * h[v] + pb;
    }
  }
  auto slopes = [&](auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
    for (int j = 0; j < LW; ++j) {
      in_order();
      if (EDGE && bit(sm, j)) initial(j);
      float f[V], rest[V], x[V];
      coefficients(j, f, rest);
      IO::get(afresh(xr[j]), x);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float da = GATE == TTT_GATE_SIGMOID ? f[v] * rest[v] : f[v];
        wv[j][v] = da * (IN == TTT_REC_PLAIN ? h[v] : h[v] - x[v]);
        h[v] = f[v] * h[v] + (IN == TTT_REC_PLAIN ? x[v] : rest[v] * x[v]);
        wv[j][v] = afresh(wv[j][v]);  // formed here, not where it is used
      }
    }
  };
  if (inner) slopes(std::false_type{});
  else slopes(std::true_type{});
  if constexpr (LINKED) {
    fold_way<V>(a, Way(i, uniform(bits.last) / (kWaves * LW), -1), c, look, e);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = 0.0f;
  }
  fold_back(wave + 1);
  const Rows<Raw, LW> dxs(a.dx, a.ldx, a.D, sizeof(E), tw, a.n), dgs(a.dg, a.ldg, a.D, sizeof(E), tw, a.n);
  auto gradients = [&](auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
    for (int j = LW - 1; j >= 0; --j) {
      in_order();
      if (EDGE && bit(em, j)) final_grad(j, e);
      float f[V], rest[V], d[V], ox[V], og[V];
      coefficients(j, f, rest);
      IO::get(afresh(dr[j]), d);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float dh = d[v] + e[v];
        ox[v] = IN == TTT_REC_PLAIN ? dh : dh * rest[v];
        og[v] = dh * wv[j][v];
        e[v] = f[v] * dh;
      }
      dxs.store(j, off, !EDGE || bit(okm, j), IO::put(ox));
      dgs.store(j, off, !EDGE || bit(okm, j), IO::put(og));
      if (EDGE && bit(sm, j) && a.dh0 && in) {
        const int s = uniform(m.start[wave * LW + j]);
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[static_cast<int64_t>(s) * a.D + c + v] = e[v];
      }
    }
  };
  if (inner) gradients(std::false_type{});
  else gradients(std::true_type{});
  pass_empty<V>(a, i, c, in, a.d_hfinal, a.dh0);
}

// A problem without tokens: every sequence's state passes through.
__global__ __launch_bounds__(kThreads) void rec_empty_kernel(RecArgs a, const float* src, float* dst) {
  const int c = static_cast<int>(blockIdx.x) * 64 + (threadIdx.x & 63);
  pass_empty<1>(a, 0, c, c < a.D, src, dst);
}

// One token for each row, a workgroup kStepThreads V channels of it: 256 rows of 4096
// bf16 (15 MB, 3 us at a copy's rate) 5.5 us; eight rows of 2048 3.2 us, which is latency.
// h[slot] <- a h[slot] + u, o = h[slot].  Rows that name
// one slot are consecutive tokens of it, in row order: the first of them does
// them all, so that the result does not depend on which workgroup comes first.  The
// search for them is B slots a workgroup: 4096 rows of 2048 bf16 58 us (without slots
// 20), 32768 rows 2.5 ms (0.16).
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
// Tiles of `tile` tokens; a problem without tokens has one, for its states.
int64_t tiles(const ttt_rec_desc& d, int tile) {
  const int64_t nt = (tokens(d) + tile - 1) / tile;
  return nt > 0 ? nt : 1;
}
constexpr int kBwdTile = kWaves * kBwdLW;
// The forward's tile: 256 tokens where that leaves eight tiles a CU, else 128.  A larger
// tile reads fewer of the others' maps: 131072 x 2048 bf16 (32 tiles of 256 a CU) takes
// 380 to 390 us with 256 and 420 with 128, 30011 x 2560 packed (9) 128 and 130; below, 4 x
// 4096 x 2048 (4) takes 61 with either, 9001 x 1001 f32 (1) 44 and 41.
int fwd_tile(const ttt_rec_desc& d) {
  const int64_t blocks = (static_cast<int64_t>(d.D) + 127) / 128;
  const int64_t nt = tiles(d, kWaves * 32);
  return nt > 1 && nt * blocks >= 8 * 256 ? kWaves * 32 : kWaves * 16;
}
// Room for either channel block width, 64 and 128.
int64_t padded_channels(const ttt_rec_desc& d) { return (static_cast<int64_t>(d.D) + 127) / 128 * 128; }

RecArgs make_args(const ttt_rec_desc& d, int V, int tile) {
  RecArgs a{};
  a.B = d.B;
  a.T = d.T;
  a.n = static_cast<int>(tokens(d));
  a.D = d.D;
  a.nt = static_cast<int>(tiles(d, tile));
  a.ncb = (d.D + 64 * V - 1) / (64 * V);
  a.Dp = static_cast<int>(padded_channels(d));
  a.ldx = d.ldx ? d.ldx : d.D;
  a.ldg = d.ldg ? d.ldg : d.D;
  return a;
}

}  // namespace

constexpr int64_t kMaxLaunch = int64_t{1} << 32;  // a launch has fewer threads

bool recurrence_step_grid_fits(const ttt_rec_desc& d) {
  return d.B * ((static_cast<int64_t>(d.D) + kStepThreads - 1) / kStepThreads) * kStepThreads < kMaxLaunch;
}

bool recurrence_grid_fits(const ttt_rec_desc& d) {
  return tiles(d, kBwdTile) * ((static_cast<int64_t>(d.D) + 63) / 64) * kThreads < kMaxLaunch;
}

namespace {

// The maps of the tiles and of the whole groups, then the counters.
size_t map_words(const ttt_rec_desc& d, int tile) {
  return static_cast<size_t>(tiles(d, tile) + tiles(d, tile) / kGroup) * padded_channels(d);
}
size_t counter_ints(const ttt_rec_desc& d) { return static_cast<size_t>((d.D + 63) / 64) * kCounterStride; }

}  // namespace

size_t recurrence_workspace(const ttt_rec_desc& d, int entry) {
  const int tile = entry == TTT_ENTRY_FWD ? fwd_tile(d) : kBwdTile;
  if (tiles(d, tile) == 1) return 0;
  return align256(map_words(d, tile) * sizeof(uint64_t)) + align256(counter_ints(d) * sizeof(int));
}

size_t recurrence_saved(const ttt_rec_desc& d) {
  return align256(static_cast<size_t>(tiles(d, kRun)) * padded_channels(d) * sizeof(float));
}

namespace {

// Lays out the workspace and clears it (a kernel, so that a graph can hold it).
hipError_t link_tiles(const ttt_rec_desc& d, int tile, RecArgs& a, void* ws, hipStream_t s) {
  a.maps = static_cast<uint64_t*>(ws);
  a.groups = a.maps + static_cast<size_t>(a.nt) * a.Dp;
  a.counters = reinterpret_cast<int*>(static_cast<char*>(ws) + align256(map_words(d, tile) * sizeof(uint64_t)));
  const int64_t n = static_cast<int64_t>(map_words(d, tile) / 2);  // Dp is even
  const int nc = static_cast<int>(counter_ints(d));
  const int64_t work = n > nc ? n : nc;
  KernelScope scope(TTT_KERNEL_REC_CLEAR, s);
  rec_clear_kernel<<<static_cast<uint32_t>((work + 255) / 256), 256, 0, s>>>(reinterpret_cast<uint4*>(ws), n, a.counters, nc);
  return hipGetLastError();
}

}  // namespace

hipError_t recurrence_fwd_launch(const ttt_rec_desc& d, const void* x, const void* gate, const float* h0, const int32_t* starts,
                                 void* o, float* h_final, void* saved, void* ws, hipStream_t s) {
  const int V = lane_channels(d.dtype, d.D, d.ldx, d.ldg);
  const int tile = fwd_tile(d);
  RecArgs a = make_args(d, V, tile);
  a.x = x; a.g = gate; a.h0 = h0; a.starts = d.packed ? starts : nullptr;
  a.o = o; a.h_final = h_final; a.ckpt = static_cast<float*>(saved);
  if (a.n == 0) {
    rec_empty_kernel<<<(d.D + 63) / 64, kThreads, 0, s>>>(a, h0, h_final);
    return hipGetLastError();
  }
  if (a.nt > 1) {
    const hipError_t e = link_tiles(d, tile, a, ws, s);
    if (e != hipSuccess) return e;
  }
  return dispatch(d, V, [&](auto e, auto v, auto gk, auto in) {
    using E = decltype(e);
    const dim3 grid(static_cast<uint32_t>(a.nt) * a.ncb);
    KernelScope scope(TTT_KERNEL_REC_FWD, s);
    if (tile == kWaves * 32) rec_fwd_kernel<E, v(), gk(), in(), 32, true><<<grid, kThreads, 0, s>>>(a);
    else if (a.nt > 1) rec_fwd_kernel<E, v(), gk(), in(), 16, true><<<grid, kThreads, 0, s>>>(a);
    else rec_fwd_kernel<E, v(), gk(), in(), 16, false><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t recurrence_bwd_launch(const ttt_rec_desc& d, const void* x, const void* gate, const float* h0, const int32_t* starts,
                                 const void* saved, const void* d_o, const float* d_hfinal, void* dx, void* dgate, float* dh0,
                                 void* ws, hipStream_t s) {
  const int V = lane_channels(d.dtype, d.D, d.ldx, d.ldg);
  RecArgs a = make_args(d, V, kBwdTile);
  a.x = x; a.g = gate; a.h0 = h0; a.starts = d.packed ? starts : nullptr;
  a.ckpt = const_cast<float*>(static_cast<const float*>(saved));
  a.d_o = d_o; a.d_hfinal = d_hfinal; a.dx = dx; a.dg = dgate; a.dh0 = dh0;
  if (a.n == 0) {
    rec_empty_kernel<<<(d.D + 63) / 64, kThreads, 0, s>>>(a, d_hfinal, dh0);
    return hipGetLastError();
  }
  if (a.nt > 1) {
    const hipError_t e = link_tiles(d, kBwdTile, a, ws, s);
    if (e != hipSuccess) return e;
  }
  return dispatch(d, V, [&](auto e, auto v, auto gk, auto in) {
    using E = decltype(e);
    const dim3 grid(static_cast<uint32_t>(a.nt) * a.ncb);
    KernelScope scope(TTT_KERNEL_REC_BWD, s);
    if (a.nt > 1) rec_bwd_kernel<E, v(), gk(), in(), kBwdLW, true><<<grid, kThreads, 0, s>>>(a);
    else rec_bwd_kernel<E, v(), gk(), in(), kBwdLW, false><<<grid, kThreads, 0, s>>>(a);
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
