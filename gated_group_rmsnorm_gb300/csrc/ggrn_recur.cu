// ggrn_recur.cu -- the gated linear recurrence over packed sequences, its form
// for single tokens and its backward pass.
//
// Per channel c, with i and r the sigmoids of the gates' logits:
//   p_t = a[c] r_t,  h_t = exp(p_t) h_{t-1} + m_t i_t x_t,  m_t = sqrt(1 - exp(2 p_t))
// and, with g_t the gradient of h_t (that of the state after the last row among
// those of later rows):
//   g_t = dout_t + e_{t+1} g_{t+1},  e_t = exp(p_t),  gradient of the first state: e_1 g_1
//   dx = g m i,  di = g m x i (1 - i),  dr = a g (h_{t-1} e r - i x e^2 r / m) (1 - r)
//   da = sum_t g (h_{t-1} e r - i x e^2 r / m),   r / m -> 0 as m -> 0
//
// Both directions are a scan of pairs (E, B): h -> E h + B.  A warp holds a few
// consecutive rows of 32 V channels and composes their pairs; the CTA's warps
// hold a tile of 64 rows and exchange theirs in shared memory; the CTAs of a
// cluster hold consecutive tiles and exchange theirs through distributed shared
// memory, one cluster barrier for all of them.  A cluster walks down (the
// gradients: up) its rows with the state in registers, so each input is read
// once and no CTA waits for another cluster.  The order of every sum is fixed.
//
// The backward pass needs the states again: the forward pass can keep the one
// before every 64th row (f32, 1/32 of a 16-bit tensor's bytes), from which each
// tile finds its own; without them a first launch makes them.
#include <cuda_runtime.h>

#include <initializer_list>
#include <type_traits>

#include "ggrn_mixer.cuh"
#include "ggrn_optin.h"

namespace ggrn {
namespace recur {

constexpr int kTile = 64;  // rows of a tile, and between the states kept
constexpr int kMaxCluster = 8;
static_assert(kTile == GGRN_RECUR_SAVED_ROWS, "a tile starts from a state that was kept");

struct Params {
  const void *x, *ig, *rg, *dout;
  const float* a;
  void *out, *dx, *dig, *drg;
  float* state;        // read where sequences resume; written by the forward pass (keep_state)
  float* saved;        // [tiles, width]: written by the forward pass, read by the backward pass
  const float* dstate; // [seqs, width]
  float* dinitial;     // [seqs, width]
  float* da;           // [segments, width]
  Seqs q;
  int64_t xs, is, rs, gs, os, dxs, dis, drs;  // row strides
  int64_t slot_stride, width;
  int segments;
  int keep_state;
  int chunk;           // bytes that the inputs' rows can be copied by: 16, 4, or an element
  int pairs;           // outputs' rows can be stored by pairs of channels
};

// V consecutive channels of T as they lie in memory.
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 2> {
  using Word = typename std::conditional<sizeof(T) == 4, uint2, uint32_t>::type;
  Word w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const Word*>(p)); }
  __device__ __forceinline__ void clear() { w = Word{}; }
  __device__ __forceinline__ void get(float* f) const {
    if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
    } else {
      Elem<T>::unpack2(w, f[0], f[1]);
    }
  }
  __device__ __forceinline__ static void put(T* p, const float* f) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
      *reinterpret_cast<uint32_t*>(p) = Elem<T>::pack2(f[0], f[1]);
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ void clear() {
    const float z = 0.0f;
    Elem<T>::store1(&w, 0, z);
  }
  __device__ __forceinline__ void get(float* f) const { f[0] = static_cast<float>(w); }
  __device__ __forceinline__ static void put(T* p, const float* f) { Elem<T>::store1(p, 0, f[0]); }
};

// ---------------------------------------------------------------------------
// Gates of a pair of elements.
//
// 16-bit T: sigmoid(z) = 1 / (1 + 2^(-z log2 e)) with the hardware's
// approximate exponential and reciprocal (both good to about 2^-22; below
// 2^-126 they give 0).  f32: the accurate functions.
//
// exp(p) - 1 comes from its series where p > -1/4 (six terms: 2^-24 of it), and
// e = 1 + that, m^2 = 1 - e^2 = -(e - 1)(2 + (e - 1)): neither loses digits to
// cancellation where decays are slow (an exponential that is off by an ulp to one
// side next to 1 is off by a thousand after a thousand rows), and slow channels
// take no second exponential.  FAST: no decay of the warp's channels is below exp(-1/4).
// ---------------------------------------------------------------------------
constexpr float kSeries = -0.25f;

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ void sigmoid2(const float* z, float* s) {
  if constexpr (Elem<T>::kExactSilu) {
    s[0] = 1.0f / (1.0f + expf(-z[0]));
    s[1] = 1.0f / (1.0f + expf(-z[1]));
  } else {
    constexpr float k = -1.4426950408889634f;
    float t0, t1;
    mul2(t0, t1, z[0], z[1], k, k);
    t0 = ex2_approx(t0), t1 = ex2_approx(t1);
    fma2(t0, t1, t0, t1, 1.0f, 1.0f, 1.0f, 1.0f);
    s[0] = rcp_approx(t0), s[1] = rcp_approx(t1);
  }
}

// exp(p) and exp(p) - 1 for p <= kSeries.
template <typename T>
__device__ __forceinline__ void beyond_series(float p, float& e, float& less) {
  if constexpr (Elem<T>::kExactSilu) {
    e = expf(p);
    less = expm1f(p);
  } else {
    e = ex2_approx(p * 1.4426950408889634f);
    less = e - 1.0f;
  }
}

// From r and the channels' a: e = exp(a r), m = sqrt(1 - e^2).
template <typename T, bool FAST>
__device__ __forceinline__ void decay2(const float* r, float a0, float a1, float* e, float* m) {
  float p[2];
  mul2(p[0], p[1], a0, a1, r[0], r[1]);
  float s0 = 1.0f / 720, s1 = 1.0f / 720, q0, q1;
  if constexpr (Elem<T>::kExactSilu) fma2(s0, s1, p[0], p[1], 1.0f / 5040, 1.0f / 5040, s0, s1);
  fma2(s0, s1, s0, s1, p[0], p[1], 1.0f / 120, 1.0f / 120);
  fma2(s0, s1, s0, s1, p[0], p[1], 1.0f / 24, 1.0f / 24);
  fma2(s0, s1, s0, s1, p[0], p[1], 1.0f / 6, 1.0f / 6);
  fma2(s0, s1, s0, s1, p[0], p[1], 0.5f, 0.5f);
  fma2(s0, s1, s0, s1, p[0], p[1], 1.0f, 1.0f);
  mul2(s0, s1, s0, s1, p[0], p[1]);  // e - 1
  fma2(e[0], e[1], s0, s1, 1.0f, 1.0f, 1.0f, 1.0f);
  if constexpr (!FAST) {
    if (!(p[0] > kSeries)) beyond_series<T>(p[0], e[0], s0);
    if (!(p[1] > kSeries)) beyond_series<T>(p[1], e[1], s1);
  }
  fma2(q0, q1, s0, s1, -1.0f, -1.0f, -2.0f, -2.0f);
  mul2(q0, q1, q0, q1, s0, s1);
  if constexpr (Elem<T>::kExactSilu) {
    m[0] = sqrtf(q0), m[1] = sqrtf(q1);
  } else {
    m[0] = sqrt_approx(q0), m[1] = sqrt_approx(q1);
  }
}

// ---------------------------------------------------------------------------
// Clusters.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void put_peer_int(const int* mine, uint32_t rank, int v) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(at),
      "r"(rank), "r"(v)
      : "memory");
}
// Stores v at the place of *mine in the shared memory of CTA `rank`.
__device__ __forceinline__ void put_peer(const float4* mine, uint32_t rank, float4 v) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(at),
      "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}

// ---------------------------------------------------------------------------
// Pairs (E, B): v -> E v + B, of a lane's two channels as (E0, E1, B0, B1).  Where
// a sequence starts (or, for gradients, ends) among the rows of a pair, nothing
// comes in from before them: E is kCut.  (Not 0: a value that is not finite would
// leave its sequence.)  CUTS: some pair may be cut.
// ---------------------------------------------------------------------------
constexpr float kCut = -1.0f;  // (decays are not negative)
template <bool CUTS>
__device__ __forceinline__ void through(const float4& s, float (&v)[2]) {
  if (CUTS && s.x == kCut) {
    v[0] = s.z, v[1] = s.w;
  } else {
    fma2(v[0], v[1], s.x, s.y, v[0], v[1], s.z, s.w);
  }
}
// s: first s, then t.
template <bool CUTS>
__device__ __forceinline__ void compose(float4& s, const float4& t) {
  if (CUTS && t.x == kCut) {
    s = t;
    return;
  }
  fma2(s.z, s.w, t.x, t.y, s.z, s.w, t.z, t.w);
  if (!CUTS || s.x != kCut) mul2(s.x, s.y, s.x, s.y, t.x, t.y);
}

// ---------------------------------------------------------------------------
// Rows and their sequences.
// ---------------------------------------------------------------------------
struct TileRows {
  uint32_t in[2], first[2], last[2];  // bits of the tile's rows
  int64_t begin, end;                 // rows of the sequence of the tile's last row
  int seq[kTile];
};

// The sequence of row r: the last one that begins at or before it.
__device__ __forceinline__ int64_t seq_of_row(const Seqs& q, int64_t r, int64_t& begin,
                                              int64_t& end) {
  int64_t s = 0;
  if (q.cu) {
    int64_t hi = q.seqs;
    while (hi - s > 1) {
      const int64_t mid = (s + hi) >> 1;
      if (__ldg(q.cu + mid) <= r) s = mid;
      else hi = mid;
    }
  } else {
    s = r / q.each;
  }
  seq_range(q, s, begin, end);
  return s;
}

// Threads 0 .. 63 of the CTA: row `tile` x 64 + thread, if it is one of [lo, hi).
__device__ __forceinline__ void place_rows(const Seqs& q, int64_t tile, int64_t lo, int64_t hi,
                                           TileRows* t) {
  const int64_t r = tile * kTile + threadIdx.x;
  bool in = false, first = false, last = false;
  int64_t begin = 0, end = 0;
  if (r >= lo && r < hi) {
    const int64_t s = seq_of_row(q, r, begin, end);
    in = r >= begin && r < end;
    first = in && r == begin;
    last = in && r == end - 1;
    t->seq[threadIdx.x] = static_cast<int>(s);
  }
  const uint32_t bi = __ballot_sync(0xffffffffu, in), bf = __ballot_sync(0xffffffffu, first),
                 bl = __ballot_sync(0xffffffffu, last);
  if ((threadIdx.x & 31) == 0) {
    t->in[threadIdx.x >> 5] = bi;
    t->first[threadIdx.x >> 5] = bf;
    t->last[threadIdx.x >> 5] = bl;
  }
  if (threadIdx.x == kTile - 1) t->begin = begin, t->end = end;
}

// What a CTA knows of its tiles' rows: those inside the sequence that it found
// last need no search.
struct Rows {
  int64_t begin = 0, end = 0;  // of that sequence
  // Whether tile `t` is whole, lies in it, and holds neither end of it.
  __device__ __forceinline__ bool inside(int64_t t) const {
    return t * kTile > begin && (t + 1) * kTile < end;
  }
};

// Rows [lo, hi) of segment z: cut where the first sequence begins that does so
// at or behind the z-th of `segments` equal shares of the rows.
__device__ __forceinline__ int64_t segment_begin(const Params& p, int z) {
  const Seqs& q = p.q;
  if (z == 0) return 0;
  if (z >= p.segments) return q.rows;
  const int64_t at = q.rows / p.segments * z;
  if (!q.cu) return (at + q.each - 1) / q.each * q.each;
  int64_t lo = 0, hi = q.seqs;  // the first of [lo, hi] that begins at or behind `at`
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (__ldg(q.cu + mid) < at) lo = mid + 1;
    else hi = mid;
  }
  if (lo >= q.seqs) return q.rows;
  const int64_t b = __ldg(q.cu + lo);
  return b < 0 ? 0 : (b > q.rows ? q.rows : b);
}

// The state that sequence s starts from, in channels c, c + 1, .. (0 where it
// starts from none).
template <int V>
__device__ __forceinline__ bool start_state(const Params& p, int64_t s, int64_t c, int n,
                                            float* h) {
  const int64_t slot = seq_slot(p.q, s);
  const bool resumes = slot >= 0 && seq_resumes(p.q, s);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = 0.0f;
    if (resumes && v < n) h[v] = p.state[slot * p.slot_stride + c + v];
  }
  return resumes;
}

// Adds to g what comes to the last row of sequence s from the state behind it.
__device__ __forceinline__ void end_gradient(const Params& p, int64_t s, int64_t c, int n,
                                             float* g) {
  if (!p.dstate) return;
#pragma unroll
  for (int v = 0; v < 2; ++v)
    if (v < n) g[v] += __ldg(p.dstate + s * p.width + c + v);
}

// Empty sequences among those of this CTA (every `of`-th 32 from the `at`-th):
// calls f(sequence) with the whole warp.
template <typename F>
__device__ __forceinline__ void each_empty(const Seqs& q, int64_t at, int64_t of, F f) {
  const int lane = threadIdx.x & 31;
  for (int64_t base = at * 32; base < q.seqs; base += of * 32) {
    int64_t b = 0, e = 1;
    if (base + lane < q.seqs) seq_range(q, base + lane, b, e);
    uint32_t m = __ballot_sync(0xffffffffu, b == e);
    for (; m; m &= m - 1) f(base + __ffs(m) - 1);
  }
}

// ---------------------------------------------------------------------------
// Tiles in shared memory: 64 rows of 64 channels of each input.
// ---------------------------------------------------------------------------
constexpr int kCols = 64;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
  }
}
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The CTA's threads start to copy tile `tile` of one input into `to`; rows
// outside [lo, hi) and channels behind the last one become zeros.
template <typename T, int THREADS>
__device__ __forceinline__ void copy_tile(T* to, const void* base, int64_t stride, int64_t c0,
                                          int64_t width, int64_t tile, int64_t lo, int64_t hi,
                                          int chunk) {
  constexpr int ES = sizeof(T);
  const T* from = static_cast<const T*>(base) + c0;
  const int64_t r0 = tile * kTile;
  const int cols = static_cast<int>(width - c0 < kCols ? width - c0 : kCols);
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if (chunk == 16) {
    constexpr int E = 16 / ES, ROW = kCols / E;  // chunks of a row
    const int c = static_cast<int>(threadIdx.x) % ROW * E;
    const int row0 = static_cast<int>(threadIdx.x) / ROW;
    const T* p = from + (r0 + row0) * stride + c;
#pragma unroll
    for (int k = 0; k < kTile * ROW / THREADS; ++k) {
      const int row = row0 + k * (THREADS / ROW);
      const bool ok = r0 + row >= lo && r0 + row < hi && c < cols;
      copy_async<16>(at + (row * kCols + c) * ES, ok ? p : from, ok ? 16 : 0);
      p += (THREADS / ROW) * stride;
    }
  } else if (chunk == 4) {
    constexpr int E = 4 / ES, ROW = kCols / E;
#pragma unroll 4
    for (int k = threadIdx.x; k < kTile * ROW; k += THREADS) {
      const int row = k / ROW, c = k % ROW * E;
      const bool ok = r0 + row >= lo && r0 + row < hi && c < cols;
      copy_async<4>(at + (row * kCols + c) * ES, ok ? from + (r0 + row) * stride + c : from,
                    !ok ? 0 : cols - c < E ? ES : 4);
    }
  } else {
#pragma unroll 4
    for (int k = threadIdx.x; k < kTile * kCols; k += THREADS) {
      const int row = k / kCols, c = k % kCols;
      T v;
      Elem<T>::store1(&v, 0, 0.0f);
      if (r0 + row >= lo && r0 + row < hi && c < cols) v = from[(r0 + row) * stride + c];
      to[k] = v;
    }
  }
}

// A lane's two channels of a row in shared memory.
template <typename T>
__device__ __forceinline__ void get2(const T* p, float* f) {
  if constexpr (sizeof(T) == 4) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
  } else {
    Elem<T>::unpack2(*reinterpret_cast<const uint32_t*>(p), f[0], f[1]);
  }
}
// Stores the first `cols` of two channels.
template <typename T>
__device__ __forceinline__ void put2(void* base, int64_t at, const float* f, int cols, bool pairs) {
  T* p = static_cast<T*>(base) + at;
  if (pairs && cols == 2) {
    Raw<T, 2>::put(p, f);
  } else {
    if (cols > 0) Elem<T>::store1(p, 0, f[0]);
    if (cols > 1) Elem<T>::store1(p, 1, f[1]);
  }
}

// ---------------------------------------------------------------------------
// Prompts.  Eight warps of eight rows each.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256, W = kThreads / 32, R = kTile / W;
static_assert(W >= kMaxCluster, "a warp to each CTA that the tile's pair goes to");

struct ForwardShared {
  float4 pair[W][32];
  float4 peer[2][kMaxCluster][32];
  int cut[2][kMaxCluster];
  TileRows rows;
};

// e and b of the warp's rows, and the pair of all of them.  INSIDE: all rows are
// those of one sequence, neither its first nor its last.
template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ void forward_rows(const Params& p, const T* tile, const float (&ac)[2],
                                             const TileRows& t, int64_t c, int cols,
                                             float (&e)[R][2], float (&b)[R][2], float4& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* mine = tile + warp * R * kCols + lane * 2;
  s = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float x[2], gi[2], gr[2], m[2];
    get2(mine + j * kCols, x);
    get2(mine + (kTile + j) * kCols, gi);
    get2(mine + (2 * kTile + j) * kCols, gr);
    sigmoid2<T>(gi, gi);
    sigmoid2<T>(gr, gr);
    decay2<T, FAST>(gr, ac[0], ac[1], e[j], m);
    mul2(m[0], m[1], m[0], m[1], gi[0], gi[1]);
    mul2(b[j][0], b[j][1], m[0], m[1], x[0], x[1]);
    if constexpr (!INSIDE) {
      const int row = warp * R + j;
      if (!(t.in[row >> 5] >> (row & 31) & 1)) {
        e[j][0] = e[j][1] = 1.0f;
        b[j][0] = b[j][1] = 0.0f;
      }
      if (t.first[row >> 5] >> (row & 31) & 1) {
        float h[2];
        if (start_state<2>(p, t.seq[row], c, cols, h))
          fma2(b[j][0], b[j][1], e[j][0], e[j][1], h[0], h[1], b[j][0], b[j][1]);
        e[j][0] = e[j][1] = kCut;
      }
    }
    compose<!INSIDE>(s, make_float4(e[j][0], e[j][1], b[j][0], b[j][1]));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) k_recur(const Params p) {
  extern __shared__ uint4 s_tile[];
  __shared__ ForwardShared sh;
  T* const tile_of = reinterpret_cast<T*>(s_tile);  // x, input gate, decay gate
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kCols, c = c0 + lane * 2;
  const int cols = c >= p.width ? 0 : p.width - c < 2 ? 1 : 2;
  if (size > 1) cluster_arrive();  // (every CTA has begun before another one writes to it)
  const int64_t lo = segment_begin(p, blockIdx.z), hi = segment_begin(p, blockIdx.z + 1);
  const int64_t tile0 = lo / kTile, tiles = hi > lo ? (hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (tiles + size - 1) / size;
  const auto fetch = [&](int64_t tile) {
    copy_tile<T, kThreads>(tile_of, p.x, p.xs, c0, p.width, tile, lo, hi, p.chunk);
    copy_tile<T, kThreads>(tile_of + kTile * kCols, p.ig, p.is, c0, p.width, tile, lo, hi, p.chunk);
    copy_tile<T, kThreads>(tile_of + 2 * kTile * kCols, p.rg, p.rs, c0, p.width, tile, lo, hi,
                           p.chunk);
  };
  if (turns > 0) fetch(tile0 + rank);
  float ac[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) ac[v] = v < cols ? __ldg(p.a + c + v) : 0.0f;
  const bool fast = __all_sync(0xffffffffu, ac[0] > kSeries && ac[1] > kSeries);
  if (size > 1) cluster_wait();

  float carry[2] = {0.0f, 0.0f};  // the state before the cluster's tiles
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t tile = tile0 + turn * size + rank;
    const int buf = turn & 1;
    const bool inside = known.inside(tile) && (tile + 1) * kTile <= hi;
    if (!inside && threadIdx.x < kTile) place_rows(p.q, tile, lo, hi, &sh.rows);
    copies_wait();
    __syncthreads();

    float e[R][2], b[R][2];
    float4 s;
    if (inside) {
      if (fast) forward_rows<T, true, true>(p, tile_of, ac, sh.rows, c, cols, e, b, s);
      else forward_rows<T, true, false>(p, tile_of, ac, sh.rows, c, cols, e, b, s);
    } else {
      forward_rows<T, false, false>(p, tile_of, ac, sh.rows, c, cols, e, b, s);
    }
    sh.pair[warp][lane] = s;
    const bool cut = !inside && (sh.rows.first[0] | sh.rows.first[1]) != 0;
    const uint32_t in = inside ? ~0u : sh.rows.in[warp * R >> 5] >> (warp * R & 31),
                   last = inside ? 0u : sh.rows.last[warp * R >> 5] >> (warp * R & 31);
    if (!inside) known.begin = sh.rows.begin, known.end = sh.rows.end;
    __syncthreads();
    if (turn + 1 < turns) fetch(tile + size);

    // the pair of the rows before this warp's in the tile, and of the whole tile
    float4 before, whole = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
    const auto fold = [&](auto cuts) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w == warp) before = whole;
        compose<decltype(cuts)::value>(whole, sh.pair[w][lane]);
      }
    };
    if (cut) fold(std::true_type());
    else fold(std::false_type());
    float h[2];
    bool cuts = cut;
    if (size > 1) {
      if (warp < size) {
        put_peer(&sh.peer[buf][rank][lane], warp, whole);
        if (lane == 0) put_peer_int(&sh.cut[buf][rank], warp, cut);
      }
      cluster_arrive();
      cluster_wait();
      for (int k = 0; k < size; ++k) cuts = cuts || sh.cut[buf][k] != 0;
      const auto pass = [&](auto some) {
        for (int k = 0; k < size; ++k) {
          if (k == rank) h[0] = carry[0], h[1] = carry[1];
          through<decltype(some)::value>(sh.peer[buf][k][lane], carry);
        }
      };
      if (cuts) pass(std::true_type());
      else pass(std::false_type());
    } else {
      h[0] = carry[0], h[1] = carry[1];
      through<true>(whole, carry);
    }
    if (p.saved && warp == 0 && tile * kTile >= lo && tile * kTile < hi) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (v < cols) p.saved[tile * p.width + c + v] = h[v];
    }
    through<true>(before, h);
    if (inside) {
      if (!p.out) continue;
      int64_t at = (tile * kTile + warp * R) * p.os + c;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        fma2(h[0], h[1], e[j][0], e[j][1], h[0], h[1], b[j][0], b[j][1]);
        put2<T>(p.out, at, h, cols, p.pairs);
        at += p.os;
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        through<true>(make_float4(e[j][0], e[j][1], b[j][0], b[j][1]), h);
        const int row = warp * R + j;
        if (p.out && (in >> j & 1))
          put2<T>(p.out, (tile * kTile + row) * p.os + c, h, cols, p.pairs);
        if (p.keep_state && (last >> j & 1)) {
          const int64_t slot = seq_slot(p.q, sh.rows.seq[row]);
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (slot >= 0 && v < cols) p.state[slot * p.slot_stride + c + v] = h[v];
        }
      }
      // (the next turn's search writes rows)
      __syncthreads();
    }
  }
  if (p.keep_state && warp == 0) {
    each_empty(p.q, static_cast<int64_t>(blockIdx.z) * size + rank,
               static_cast<int64_t>(size) * p.segments, [&](int64_t s) {
                 const int64_t slot = seq_slot(p.q, s);
                 if (slot < 0 || seq_resumes(p.q, s)) return;
                 for (int v = 0; v < cols; ++v) p.state[slot * p.slot_stride + c + v] = 0.0f;
               });
  }
}

// ---------------------------------------------------------------------------
// Gradients.  The cluster's tiles go from the last rows to the first; rank 0 has
// the last of them.
// ---------------------------------------------------------------------------
struct BackwardShared {
  float4 down[W][32];  // pairs of states
  float4 up[W][32];    // pairs of gradients
  float4 peer[2][kMaxCluster][32];
  int cut[2][kMaxCluster];
  TileRows rows;
};

// What the warp's rows need again, and their pairs.
struct BackwardRows {
  float e[R][2], m[R][2], si[R][2], sr[R][2];
};
template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ void backward_rows(const Params& p, const T* tile, const float (&ac)[2],
                                              const TileRows& t, int64_t c, int cols,
                                              BackwardRows& k, float4& down, float4& up) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* mine = tile + warp * R * kCols + lane * 2;
  down = up = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float x[2], b[2];
    get2(mine + j * kCols, x);
    get2(mine + (kTile + j) * kCols, k.si[j]);
    get2(mine + (2 * kTile + j) * kCols, k.sr[j]);
    sigmoid2<T>(k.si[j], k.si[j]);
    sigmoid2<T>(k.sr[j], k.sr[j]);
    decay2<T, FAST>(k.sr[j], ac[0], ac[1], k.e[j], k.m[j]);
    mul2(b[0], b[1], k.m[j][0], k.m[j][1], k.si[j][0], k.si[j][1]);
    mul2(b[0], b[1], b[0], b[1], x[0], x[1]);
    if constexpr (!INSIDE) {
      const int row = warp * R + j;
      if (!(t.in[row >> 5] >> (row & 31) & 1)) {
        k.e[j][0] = k.e[j][1] = 1.0f;
        b[0] = b[1] = 0.0f;
      }
      if (t.first[row >> 5] >> (row & 31) & 1) {
        float h[2];
        start_state<2>(p, t.seq[row], c, cols, h);
        fma2(b[0], b[1], k.e[j][0], k.e[j][1], h[0], h[1], b[0], b[1]);
        down = make_float4(kCut, kCut, b[0], b[1]);
        continue;
      }
    }
    compose<!INSIDE>(down, make_float4(k.e[j][0], k.e[j][1], b[0], b[1]));
  }
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    float g[2];
    get2(mine + (3 * kTile + j) * kCols, g);
    if constexpr (!INSIDE) {
      const int row = warp * R + j;
      if (!(t.in[row >> 5] >> (row & 31) & 1)) continue;
      if (t.last[row >> 5] >> (row & 31) & 1) {
        end_gradient(p, t.seq[row], c, cols, g);
        mul2(g[0], g[1], g[0], g[1], k.e[j][0], k.e[j][1]);
        up = make_float4(kCut, kCut, g[0], g[1]);
        continue;
      }
    }
    mul2(g[0], g[1], g[0], g[1], k.e[j][0], k.e[j][1]);
    compose<!INSIDE>(up, make_float4(k.e[j][0], k.e[j][1], g[0], g[1]));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_recur_backward(const Params p, int stages) {
  extern __shared__ uint4 s_tile[];
  __shared__ BackwardShared sh;
  constexpr int kInput = kTile * kCols;  // elements of an input's tile
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kCols, c = c0 + lane * 2;
  const int cols = c >= p.width ? 0 : p.width - c < 2 ? 1 : 2;
  cluster_arrive();  // (every CTA has begun before another one writes to it)
  const int64_t lo = segment_begin(p, blockIdx.z), hi = segment_begin(p, blockIdx.z + 1);
  const int64_t tile0 = lo / kTile, tiles = hi > lo ? (hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (tiles + size - 1) / size;
  const int64_t top = tile0 + tiles - 1;  // the last tile
  const auto fetch = [&](int64_t tile, T* to) {
    copy_tile<T, kThreads>(to, p.x, p.xs, c0, p.width, tile, lo, hi, p.chunk);
    copy_tile<T, kThreads>(to + kInput, p.ig, p.is, c0, p.width, tile, lo, hi, p.chunk);
    copy_tile<T, kThreads>(to + 2 * kInput, p.rg, p.rs, c0, p.width, tile, lo, hi, p.chunk);
    copy_tile<T, kThreads>(to + 3 * kInput, p.dout, p.gs, c0, p.width, tile, lo, hi, p.chunk);
  };
  T* const ring = reinterpret_cast<T*>(s_tile);
  if (turns > 0) fetch(top - rank, ring);
  float ac[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) ac[v] = v < cols ? __ldg(p.a + c + v) : 0.0f;
  const bool fast = __all_sync(0xffffffffu, ac[0] > kSeries && ac[1] > kSeries);
  cluster_wait();

  float carry[2] = {0.0f, 0.0f}, da[2] = {0.0f, 0.0f};
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t tile = top - (turn * size + rank);
    const int buf = turn & 1;
    const T* const mine = ring + (stages == 2 ? buf : 0) * 4 * kInput;
    const bool inside = tile * kTile >= lo && known.inside(tile);
    if (!inside && threadIdx.x < kTile) place_rows(p.q, tile, lo, hi, &sh.rows);
    float h[2];  // the state before the tile, as it was kept
#pragma unroll
    for (int v = 0; v < 2; ++v)
      h[v] = tile * kTile >= lo && v < cols ? __ldg(p.saved + tile * p.width + c + v) : 0.0f;
    copies_wait();
    __syncthreads();
    if (stages == 2 && turn + 1 < turns) fetch(tile - size, ring + (buf ^ 1) * 4 * kInput);

    BackwardRows k;
    {
      float4 down, up;
      if (inside) {
        if (fast) backward_rows<T, true, true>(p, mine, ac, sh.rows, c, cols, k, down, up);
        else backward_rows<T, true, false>(p, mine, ac, sh.rows, c, cols, k, down, up);
      } else {
        backward_rows<T, false, false>(p, mine, ac, sh.rows, c, cols, k, down, up);
      }
      sh.down[warp][lane] = down;
      sh.up[warp][lane] = up;
    }
    const uint32_t in = inside ? ~0u : sh.rows.in[warp * R >> 5] >> (warp * R & 31),
                   first = inside ? 0u : sh.rows.first[warp * R >> 5] >> (warp * R & 31),
                   last = inside ? 0u : sh.rows.last[warp * R >> 5] >> (warp * R & 31);
    const bool cut = !inside && (sh.rows.last[0] | sh.rows.last[1]) != 0;
    if (!inside) {  // (of the tile's first row: its tiles come next)
      int64_t b, e;
      known.begin = known.end = 0;
      if (tile * kTile >= lo && tile * kTile < hi) {
        seq_range(p.q, sh.rows.seq[0], b, e);
        known.begin = b, known.end = e;
      }
    }
    __syncthreads();
    // the pair of the rows behind this warp's in the tile, and of the whole tile
    float4 behind, whole = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
    const auto fold = [&](auto cuts) {
#pragma unroll
      for (int w = W - 1; w >= 0; --w) {
        if (w == warp) behind = whole;
        compose<decltype(cuts)::value>(whole, sh.up[w][lane]);
      }
    };
    if (cut) fold(std::true_type());
    else fold(std::false_type());
    if (size > 1) {
      if (warp < size) {
        put_peer(&sh.peer[buf][rank][lane], warp, whole);
        if (lane == 0) put_peer_int(&sh.cut[buf][rank], warp, cut);
      }
      cluster_arrive();
    }
    // the states before each row, meanwhile
    float hp[R][2];
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
      if (w < warp) {
        if (inside) through<false>(sh.down[w][lane], h);
        else through<true>(sh.down[w][lane], h);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (first >> j & 1) start_state<2>(p, sh.rows.seq[warp * R + j], c, cols, h);
      float x[2], b[2];
      get2(mine + (warp * R + j) * kCols + lane * 2, x);
      mul2(b[0], b[1], k.m[j][0], k.m[j][1], k.si[j][0], k.si[j][1]);
      mul2(b[0], b[1], b[0], b[1], x[0], x[1]);
      hp[j][0] = h[0], hp[j][1] = h[1];
      if (in >> j & 1) fma2(h[0], h[1], k.e[j][0], k.e[j][1], h[0], h[1], b[0], b[1]);
    }

    // the gradient that comes to this warp's last row from the rows behind it
    float gc[2];
    if (size > 1) {
      cluster_wait();
      bool cuts = false;
      for (int q = 0; q < size; ++q) cuts = cuts || sh.cut[buf][q] != 0;
      const auto pass = [&](auto some) {
        for (int q = 0; q < size; ++q) {
          if (q == rank) gc[0] = carry[0], gc[1] = carry[1];
          through<decltype(some)::value>(sh.peer[buf][q][lane], carry);
        }
      };
      if (cuts) pass(std::true_type());
      else pass(std::false_type());
    } else {
      gc[0] = carry[0], gc[1] = carry[1];
      through<true>(whole, carry);
    }
    through<true>(behind, gc);
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const int row = warp * R + j;
      const int64_t r = tile * kTile + row;
      float g[2], x[2], dx[2], di[2], dr[2], t1[2], t2[2];
      get2(mine + row * kCols + lane * 2, x);
      get2(mine + 3 * kInput + row * kCols + lane * 2, g);
      const float(&e)[2] = k.e[j], (&m)[2] = k.m[j], (&si)[2] = k.si[j], (&sr)[2] = k.sr[j];
      if (last >> j & 1) end_gradient(p, sh.rows.seq[row], c, cols, g);
      else fma2(g[0], g[1], g[0], g[1], 1.0f, 1.0f, gc[0], gc[1]);
      // dx = g m i,  di = dx x (1 - i)
      mul2(dx[0], dx[1], m[0], m[1], si[0], si[1]);
      mul2(dx[0], dx[1], dx[0], dx[1], g[0], g[1]);
      fma2(di[0], di[1], si[0], si[1], -1.0f, -1.0f, 1.0f, 1.0f);
      mul2(di[0], di[1], di[0], di[1], x[0], x[1]);
      mul2(di[0], di[1], di[0], di[1], dx[0], dx[1]);
      // g (h e r - i x e^2 r / m)
      float over[2];
#pragma unroll
      for (int v = 0; v < 2; ++v)
        over[v] = m[v] > 0.0f ? (Elem<T>::kExactSilu ? 1.0f / m[v] : rcp_approx(m[v])) : 0.0f;
      mul2(t2[0], t2[1], si[0], si[1], x[0], x[1]);
      mul2(t2[0], t2[1], t2[0], t2[1], e[0], e[1]);
      mul2(t2[0], t2[1], t2[0], t2[1], over[0], over[1]);
      fma2(t1[0], t1[1], t2[0], t2[1], -1.0f, -1.0f, hp[j][0], hp[j][1]);
      mul2(t2[0], t2[1], e[0], e[1], sr[0], sr[1]);
      mul2(t1[0], t1[1], t1[0], t1[1], t2[0], t2[1]);
      mul2(t1[0], t1[1], t1[0], t1[1], g[0], g[1]);
      fma2(dr[0], dr[1], sr[0], sr[1], -1.0f, -1.0f, 1.0f, 1.0f);
      mul2(dr[0], dr[1], dr[0], dr[1], ac[0], ac[1]);
      mul2(dr[0], dr[1], dr[0], dr[1], t1[0], t1[1]);
      if (in >> j & 1) {
        fma2(da[0], da[1], t1[0], t1[1], 1.0f, 1.0f, da[0], da[1]);
        mul2(gc[0], gc[1], e[0], e[1], g[0], g[1]);
      } else {  // a row of no sequence
#pragma unroll
        for (int v = 0; v < 2; ++v) dx[v] = di[v] = dr[v] = 0.0f;
      }
      if (inside || (r >= lo && r < hi)) {
        put2<T>(p.dx, r * p.dxs + c, dx, cols, p.pairs);
        put2<T>(p.dig, r * p.dis + c, di, cols, p.pairs);
        put2<T>(p.drg, r * p.drs + c, dr, cols, p.pairs);
      }
      if (p.dinitial && (first >> j & 1)) {
        const int64_t s = sh.rows.seq[row];
        const bool resumes = seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (v < cols) p.dinitial[s * p.width + c + v] = resumes ? gc[v] : 0.0f;
      }
    }
    // (the next turn's search writes rows, its copies the tile)
    if (!inside || stages == 1) __syncthreads();
    if (stages == 1 && turn + 1 < turns) fetch(tile - size, ring);
  }
  if (p.dinitial && warp == 0) {
    each_empty(p.q, static_cast<int64_t>(blockIdx.z) * size + rank,
               static_cast<int64_t>(size) * p.segments, [&](int64_t s) {
                 const bool keep = p.dstate && seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
                 for (int v = 0; v < cols; ++v) {
                   const int64_t k = s * p.width + c + v;
                   p.dinitial[k] = keep ? __ldg(p.dstate + k) : 0.0f;
                 }
               });
  }
  // da: the warps' sums, then the CTAs' in rank 0
  __syncthreads();
  sh.up[warp][lane] = make_float4(da[0], da[1], 0.0f, 0.0f);
  __syncthreads();
  if (warp == 0) {
    float4 t = sh.up[0][lane];
    for (int w = 1; w < W; ++w) t.x += sh.up[w][lane].x, t.y += sh.up[w][lane].y;
    put_peer(&sh.peer[turns & 1][rank][lane], 0, t);
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0 && warp == 0) {
    float t[2] = {0.0f, 0.0f};
    for (int q = 0; q < size; ++q) {
      t[0] += sh.peer[turns & 1][q][lane].x;
      t[1] += sh.peer[turns & 1][q][lane].y;
    }
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (v < cols) p.da[blockIdx.z * p.width + c + v] = t[v];
  }
}

// out[c] = the sum of in[k, c] over the segments.
__global__ void __launch_bounds__(256) k_recur_sum(const float* in, float* out, int64_t width,
                                                   int segments) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= width) return;
  float t = 0.0f;
  for (int k = 0; k < segments; ++k) t += in[k * width + c];
  out[c] = t;
}

// ---------------------------------------------------------------------------
// One row of each sequence.
// ---------------------------------------------------------------------------
template <typename T, int V>
__global__ void __launch_bounds__(128) k_recur_step(const Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V;
  const int64_t row = blockIdx.x;
  const int64_t slot = seq_slot(p.q, row);
  if (c >= p.width || slot < 0) return;
  // (two elements at a time; the second is the first again where there is one)
  constexpr int N = V == 1 ? 2 : V;
  float x[N], gi[N], gr[N], ac[N], h[N], e[N], m[N];
  float* state = p.state + slot * p.slot_stride + c;
  Raw<T, V> xr, ir, rr;
  xr.load(static_cast<const T*>(p.x) + row * p.xs + c);
  ir.load(static_cast<const T*>(p.ig) + row * p.is + c);
  rr.load(static_cast<const T*>(p.rg) + row * p.rs + c);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ac[v] = __ldg(p.a + c + v);
    h[v] = state[v];
  }
  xr.get(x), ir.get(gi), rr.get(gr);
  if constexpr (V == 1) x[1] = x[0], gi[1] = gi[0], gr[1] = gr[0], ac[1] = ac[0], h[1] = h[0];
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    sigmoid2<T>(gi + k, gi + k);
    sigmoid2<T>(gr + k, gr + k);
    decay2<T, false>(gr + k, ac[k], ac[k + 1], e + k, m + k);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = fmaf(e[v], h[v], m[v] * gi[v] * x[v]);
    state[v] = h[v];
  }
  Raw<T, V>::put(static_cast<T*>(p.out) + row * p.os + c, h);
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
// How the tiles of a call are shared out: CTAs of a cluster, and segments.
struct Split {
  int cluster = 1, segments = 1;
};

Split split_rows(int64_t rows, int64_t seqs, int64_t blocks, int resident) {
  Split s;
  const int64_t tiles = (rows + kTile - 1) / kTile, sms = device_sms();
  const int64_t most = tiles < kMaxCluster ? (tiles < 1 ? 1 : tiles) : kMaxCluster;
  // the cluster whose fullest SM has least to do; the smaller one of two alike
  double best = 1e30;
  for (int64_t k = 1; k <= most; ++k) {
    const int64_t ctas = blocks * k;
    const int64_t per_sm = (ctas + sms - 1) / sms;
    const double cost = static_cast<double>(per_sm) / static_cast<double>(k);
    if (cost < best * 0.98) best = cost, s.cluster = static_cast<int>(k);
  }
  const int64_t want = sms * resident / (blocks * s.cluster);
  int64_t parts = want < seqs ? want : seqs;
  if (parts > tiles / s.cluster) parts = tiles / s.cluster;
  if (parts > 1) s.segments = static_cast<int>(parts < 65535 ? parts : 65535);
  return s;
}

template <typename... P, typename... A>
int launch_cluster(void (*kernel)(P...), int64_t blocks, Split s, int smem, cudaStream_t stream,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.cluster), static_cast<unsigned>(blocks),
                     static_cast<unsigned>(s.segments));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(s.cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  return GGRN_OK;
}

int64_t blocks_of(int64_t width) { return (width + kCols - 1) / kCols; }

template <typename T>
int launch_forward(Params& p, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width);
  const Split k = split_rows(p.q.rows, p.q.seqs, blocks, sizeof(T) == 2 ? 4 : 3);
  p.segments = k.segments;
  constexpr int kSmem = 3 * kTile * kCols * sizeof(T);
  const cudaError_t e = allow_shared_memory<k_recur<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  return launch_cluster(k_recur<T>, blocks, k, kSmem, s, p);
}
template <typename T>
int launch_backward(Params& p, float* sums, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width);
  const Split k = split_rows(p.q.rows, p.q.seqs, blocks, 2);
  p.segments = k.segments;
  float* const da = p.da;
  if (k.segments > 1) p.da = sums;
  // two tiles of 16-bit types in shared memory, one of f32
  constexpr int kStages = sizeof(T) == 2 ? 2 : 1;
  constexpr int kSmem = kStages * 4 * kTile * kCols * sizeof(T);
  const cudaError_t e = allow_shared_memory<k_recur_backward<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  const int st = launch_cluster(k_recur_backward<T>, blocks, k, kSmem, s, p, kStages);
  if (st != GGRN_OK || k.segments == 1) return st;
  return mixer::launch(k_recur_sum, dim3(static_cast<unsigned>((p.width + 255) / 256)), 256, 0, s,
                       static_cast<const float*>(sums), da, p.width, k.segments);
}
template <typename T, int V>
int launch_step(const Params& p, cudaStream_t s) {
  const int64_t gy = (p.width + 128 * V - 1) / (128 * V);
  if (p.q.rows > INT32_MAX) return GGRN_ERR_UNSUPPORTED;
  return mixer::launch(k_recur_step<T, V>,
                       dim3(static_cast<unsigned>(p.q.rows), static_cast<unsigned>(gy)), 128, 0, s,
                       p);
}

// Widths that a grid's second axis holds (a block of channels each, or 128 in the
// step form).
constexpr int64_t kMostColumns = int64_t{65535} * 32;

struct Matrix {
  const void* p;
  int64_t stride;
};
// Pairs of channels: every row of every matrix starts on one.
bool pairs(int64_t rows, int es, std::initializer_list<Matrix> ms) {
  for (const Matrix& m : ms)
    if (!mixer::aligned_to(m.p, 2 * es) || (rows > 1 && m.stride % 2)) return false;
  return true;
}

// Bytes that every row of every matrix can be copied by.
int chunk_of(int64_t rows, int64_t width, int es, std::initializer_list<Matrix> ms) {
  for (int bytes : {16, 4}) {
    bool fits = bytes == 4 || width * es % 16 == 0;
    for (const Matrix& m : ms)
      fits = fits && mixer::aligned_to(m.p, bytes) && (rows <= 1 || m.stride * es % bytes == 0);
    if (fits) return bytes;
  }
  return es;
}

int check_sizes(int dtype, int64_t rows, int64_t width) {
  if (dtype != kF32 && dtype != kF16 && dtype != kBF16) return GGRN_ERR_DTYPE;
  if (width <= 0) return GGRN_ERR_SHAPE;
  if (width > int64_t{1} << 40) return GGRN_ERR_SHAPE;
  if (width > kMostColumns) return GGRN_ERR_UNSUPPORTED;
  // the states kept, and gradients of states, fit in int64
  if (rows > (int64_t{1} << 60) / width) return GGRN_ERR_SHAPE;
  return GGRN_OK;
}

int check(const ggrn_recur_call& c, bool step, Params* p) {
  int st = check_sizes(c.dtype, c.rows, c.width);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  st = mixer::check_seqs(c.rows, c.seqs, c.cu_seqlens, c.state, c.slots, c.resume, c.state_slots,
                         c.width, c.state_slot_stride, step, &p->q);
  if (st != GGRN_OK) return st;
  mixer::Buffer x, ig, rg, out, state;
  if (!mixer::extent(c.x, c.rows, c.width, c.x_row_stride, es, &x) ||
      !mixer::extent(c.input_gate, c.rows, c.width, c.input_gate_row_stride, es, &ig) ||
      !mixer::extent(c.decay_gate, c.rows, c.width, c.decay_gate_row_stride, es, &rg) ||
      !mixer::extent(c.out, c.rows, c.width, c.out_row_stride, es, &out) ||
      !mixer::extent(c.state, c.state ? c.state_slots : 0, c.width, c.state_slot_stride, 4,
                     &state))
    return GGRN_ERR_SHAPE;
  if (c.rows == 0 && (!c.state || p->q.seqs == 0)) return GGRN_OK;
  if (!c.a || (c.rows > 0 && (!c.x || !c.input_gate || !c.decay_gate || !c.out)))
    return GGRN_ERR_NULL;
  float* const saved_p = step ? nullptr : c.saved;
  for (const void* q : {c.x, c.input_gate, c.decay_gate, static_cast<const void*>(c.out)})
    if (!mixer::aligned_to(q, es)) return GGRN_ERR_ALIGN;
  if (!mixer::aligned_to(c.a, 4) || !mixer::aligned_to(c.state, 4) ||
      !mixer::aligned_to(saved_p, 4))
    return GGRN_ERR_ALIGN;
  const mixer::Buffer a = {c.a, c.width * 4}, cu = {p->q.cu, (p->q.seqs + 1) * 4},
                      slots = {p->q.slots, p->q.seqs * 4}, res = {p->q.resume, p->q.seqs},
                      saved = {saved_p, (c.rows + kTile - 1) / kTile * c.width * 4};
  for (const mixer::Buffer& o : {out, state, saved})
    for (const mixer::Buffer& i : {x, ig, rg, a, cu, slots, res})
      if (mixer::overlap(o, i)) return GGRN_ERR_OVERLAP;
  if (mixer::overlap(out, state) || mixer::overlap(out, saved) || mixer::overlap(state, saved))
    return GGRN_ERR_OVERLAP;
  p->x = c.x;
  p->ig = c.input_gate;
  p->rg = c.decay_gate;
  p->a = c.a;
  p->out = c.out;
  p->state = c.state;
  p->saved = saved_p;
  const bool many = c.rows > 1;
  p->xs = many ? c.x_row_stride : 0;
  p->is = many ? c.input_gate_row_stride : 0;
  p->rs = many ? c.decay_gate_row_stride : 0;
  p->os = many ? c.out_row_stride : 0;
  p->slot_stride = c.state_slots > 1 ? c.state_slot_stride : 0;
  p->width = c.width;
  p->keep_state = c.state != nullptr;
  return GGRN_OK;
}

int run(const ggrn_recur_call* call, bool step, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_recur_call& c = *call;
  Params p = {};
  const int st = check(c, step, &p);
  if (st != GGRN_OK || (c.rows == 0 && (step || !c.state || p.q.seqs == 0))) return st;
  const int es = mixer::elem_bytes(c.dtype);
  const bool two = c.width % 2 == 0 && pairs(c.rows, es, {{c.x, p.xs}, {c.input_gate, p.is},
                                                          {c.decay_gate, p.rs}, {c.out, p.os}});
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.chunk = chunk_of(c.rows, c.width, es, {{c.x, p.xs}, {c.input_gate, p.is}, {c.decay_gate, p.rs}});
  p.pairs = pairs(c.rows, es, {{c.out, p.os}});
  if (step) {
    if (c.dtype == kF32) return two ? launch_step<float, 2>(p, s) : launch_step<float, 1>(p, s);
    if (c.dtype == kF16) return two ? launch_step<__half, 2>(p, s) : launch_step<__half, 1>(p, s);
    return two ? launch_step<__nv_bfloat16, 2>(p, s) : launch_step<__nv_bfloat16, 1>(p, s);
  }
  if (c.dtype == kF32) return launch_forward<float>(p, s);
  if (c.dtype == kF16) return launch_forward<__half>(p, s);
  return launch_forward<__nv_bfloat16>(p, s);
}

// Workspace of the backward pass: the states that were not kept, then the
// segments' sums of da.
struct Space {
  int64_t saved, sums;  // bytes
};
Space space_of(const ggrn_recur_backward_call& c) {
  const int64_t tiles = (c.rows + kTile - 1) / kTile;
  Space s = {c.saved ? 0 : tiles * c.width * 4, 0};
  s.saved = (s.saved + 15) / 16 * 16;
  const int64_t most = split_rows(c.rows, c.seqs, blocks_of(c.width), 2).segments;
  if (most > 1) s.sums = most * c.width * 4;
  return s;
}

int check_backward(const ggrn_recur_backward_call& c, Params* p) {
  int st = check_sizes(c.dtype, c.rows, c.width);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  st = mixer::check_seqs(c.rows, c.seqs, c.cu_seqlens, c.state, c.slots, c.resume, c.state_slots,
                         c.width, c.state_slot_stride, false, &p->q);
  if (st != GGRN_OK) return st;
  if (p->q.seqs > (int64_t{1} << 60) / c.width) return GGRN_ERR_SHAPE;
  const struct { const void* p; int64_t stride; } mats[7] = {
      {c.dout, c.dout_row_stride}, {c.x, c.x_row_stride},
      {c.input_gate, c.input_gate_row_stride}, {c.decay_gate, c.decay_gate_row_stride},
      {c.dx, c.dx_row_stride}, {c.dinput_gate, c.dinput_gate_row_stride},
      {c.ddecay_gate, c.ddecay_gate_row_stride}};
  mixer::Buffer b[7], state;
  for (int k = 0; k < 7; ++k)
    if (!mixer::extent(mats[k].p, c.rows, c.width, mats[k].stride, es, &b[k]))
      return GGRN_ERR_SHAPE;
  if (!mixer::extent(c.state, c.state ? c.state_slots : 0, c.width, c.state_slot_stride, 4, &state))
    return GGRN_ERR_SHAPE;
  if (!c.a || !c.da) return GGRN_ERR_NULL;
  for (int k = 0; k < 7; ++k) {
    if (c.rows > 0 && !mats[k].p) return GGRN_ERR_NULL;
    if (!mixer::aligned_to(mats[k].p, es)) return GGRN_ERR_ALIGN;
  }
  for (const void* q : {static_cast<const void*>(c.a), static_cast<const void*>(c.da),
                        static_cast<const void*>(c.state), static_cast<const void*>(c.saved),
                        static_cast<const void*>(c.dstate), static_cast<const void*>(c.dinitial)})
    if (!mixer::aligned_to(q, 4)) return GGRN_ERR_ALIGN;
  const Space need = space_of(c);
  if (need.saved + need.sums > 0) {
    if (!c.workspace) return GGRN_ERR_NULL;
    if (!mixer::aligned_to(c.workspace, 16)) return GGRN_ERR_ALIGN;
    if (c.workspace_bytes < need.saved + need.sums) return GGRN_ERR_ARG;
  }
  const int64_t kept = (c.rows + kTile - 1) / kTile * c.width * 4, ends = p->q.seqs * c.width * 4;
  const auto matrix = [&](int k) {
    return mixer::columns(b[k], c.rows, c.width, mats[k].stride, es);
  };
  const auto vector = [](const void* q, int64_t n) { return mixer::Columns{{q, n}, 0, 0}; };
  if (mixer::outputs_overlap(
          {matrix(4), matrix(5), matrix(6), vector(c.da, c.width * 4), vector(c.dinitial, ends),
           vector(c.workspace, need.saved + need.sums)},
          {matrix(0), matrix(1), matrix(2), matrix(3), mixer::Columns{state, 0, 0},
           vector(c.a, c.width * 4), vector(c.saved, kept), vector(c.dstate, ends),
           vector(p->q.cu, (p->q.seqs + 1) * 4), vector(p->q.slots, p->q.seqs * 4),
           vector(p->q.resume, p->q.seqs)}))
    return GGRN_ERR_OVERLAP;
  const bool many = c.rows > 1;
  p->x = c.x;
  p->ig = c.input_gate;
  p->rg = c.decay_gate;
  p->dout = c.dout;
  p->a = c.a;
  p->dx = c.dx;
  p->dig = c.dinput_gate;
  p->drg = c.ddecay_gate;
  p->da = c.da;
  p->state = const_cast<float*>(c.state);
  p->dstate = c.dstate;
  p->dinitial = c.dinitial;
  p->saved = const_cast<float*>(c.saved);
  p->gs = many ? c.dout_row_stride : 0;
  p->xs = many ? c.x_row_stride : 0;
  p->is = many ? c.input_gate_row_stride : 0;
  p->rs = many ? c.decay_gate_row_stride : 0;
  p->dxs = many ? c.dx_row_stride : 0;
  p->dis = many ? c.dinput_gate_row_stride : 0;
  p->drs = many ? c.ddecay_gate_row_stride : 0;
  p->slot_stride = c.state_slots > 1 ? c.state_slot_stride : 0;
  p->width = c.width;
  return GGRN_OK;
}

template <typename T>
int backward(Params& p, const Space& need, void* workspace, cudaStream_t s) {
  if (!p.saved && p.q.rows > 0) {
    Params f = p;
    p.saved = f.saved = static_cast<float*>(workspace);
    const int st = launch_forward<T>(f, s);
    if (st != GGRN_OK) return st;
  }
  float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + need.saved);
  return launch_backward<T>(p, sums, s);
}

int run_backward(const ggrn_recur_backward_call* call, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_recur_backward_call& c = *call;
  Params p = {};
  const int st = check_backward(c, &p);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  p.chunk = chunk_of(c.rows, c.width, es, {{c.dout, p.gs}, {c.x, p.xs}, {c.input_gate, p.is},
                                           {c.decay_gate, p.rs}});
  p.pairs = pairs(c.rows, es, {{c.dx, p.dxs}, {c.dinput_gate, p.dis}, {c.ddecay_gate, p.drs}});
  const Space need = space_of(c);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* const w = c.workspace;
  if (c.dtype == kF32) return backward<float>(p, need, w, s);
  if (c.dtype == kF16) return backward<__half>(p, need, w, s);
  return backward<__nv_bfloat16>(p, need, w, s);
}

}  // namespace recur

int check_recur(const ggrn_recur_call& c, bool step) {
  recur::Params p = {};
  return recur::check(c, step, &p);
}

}  // namespace ggrn

extern "C" int ggrn_recur(const ggrn_recur_call* call, void* cuda_stream) {
  return ggrn::recur::run(call, false, cuda_stream);
}
extern "C" int ggrn_recur_step(const ggrn_recur_call* call, void* cuda_stream) {
  return ggrn::recur::run(call, true, cuda_stream);
}
extern "C" int ggrn_recur_backward(const ggrn_recur_backward_call* call, void* cuda_stream) {
  return ggrn::recur::run_backward(call, cuda_stream);
}
extern "C" int64_t ggrn_recur_backward_workspace_bytes(const ggrn_recur_backward_call* call) {
  if (!call || ggrn::recur::check_sizes(call->dtype, call->rows, call->width) != GGRN_OK ||
      !ggrn::mixer::counts_ok(call->rows, call->seqs, call->cu_seqlens != nullptr))
    return 0;
  const ggrn::recur::Space s = ggrn::recur::space_of(*call);
  return s.saved + s.sums;
}
