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
// Stores a pair at the place of *mine in the shared memory of CTA `rank`.
__device__ __forceinline__ void put_peer(const float2* mine, uint32_t rank, float2 v) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(at),
      "r"(rank), "f"(v.x), "f"(v.y)
      : "memory");
}

// ---------------------------------------------------------------------------
// Pairs (E, B): v -> E v + B.  Where a sequence starts (or, for gradients, ends)
// among the rows of a pair, nothing comes in from before them: E is kCut.
// ---------------------------------------------------------------------------
constexpr float kCut = -1.0f;  // (decays are not negative)
__device__ __forceinline__ float through(float2 s, float v) {
  return s.x == kCut ? s.y : fmaf(s.x, v, s.y);
}
// First `s`, then `t`.
__device__ __forceinline__ float2 compose(float2 s, float2 t) {
  if (t.x == kCut) return t;
  return make_float2(s.x == kCut ? kCut : s.x * t.x, fmaf(t.x, s.y, t.y));
}

// ---------------------------------------------------------------------------
// Rows and their sequences.
// ---------------------------------------------------------------------------
struct TileRows {
  uint32_t in[2], first[2], last[2];  // bits of the tile's rows
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
  if (r >= lo && r < hi) {
    int64_t begin, end;
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
}

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
// Prompts.
// ---------------------------------------------------------------------------
template <typename T, int V>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) k_recur(const Params p) {
  constexpr int W = 8, R = kTile / W, N = R * V, C = 32 * V;
  __shared__ float2 s_warp[W][C];
  __shared__ float2 s_peer[2][kMaxCluster][C];
  __shared__ TileRows s_rows[2];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * V;
  const int cols = c >= p.width ? 0 : static_cast<int>(p.width - c < V ? p.width - c : V);
  float ac[V];
  bool fast = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ac[v] = v < cols ? __ldg(p.a + c + v) : 0.0f;
    fast = fast && ac[v] > kSeries;
  }
  fast = __all_sync(0xffffffffu, fast);
  const int64_t lo = segment_begin(p, blockIdx.z), hi = segment_begin(p, blockIdx.z + 1);
  const int64_t tile0 = lo / kTile, tiles = hi > lo ? (hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (tiles + size - 1) / size;

  const T* x = static_cast<const T*>(p.x) + c;
  const T* ig = static_cast<const T*>(p.ig) + c;
  const T* rg = static_cast<const T*>(p.rg) + c;
  T* out = static_cast<T*>(p.out) + c;
  Raw<T, V> xr[R], ir[R], rr[R];
  auto fetch = [&](int64_t tile) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = tile * kTile + warp * R + j;
      if (cols == V && r >= lo && r < hi) {
        xr[j].load(x + r * p.xs);
        ir[j].load(ig + r * p.is);
        rr[j].load(rg + r * p.rs);
      } else {
        xr[j].clear(), ir[j].clear(), rr[j].clear();
      }
    }
    if (threadIdx.x < kTile) place_rows(p.q, tile, lo, hi, &s_rows[(tile - tile0) / size & 1]);
  };

  float carry[V] = {};  // the state before the cluster's tiles
  cluster_arrive();     // (every CTA has begun before another one writes to it)
  if (turns > 0) fetch(tile0 + rank);
  cluster_wait();
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t tile = tile0 + turn * size + rank;
    const int buf = turn & 1;
    __syncthreads();
    const int shift = warp * R & 31;
    const uint32_t in = s_rows[buf].in[warp * R >> 5] >> shift,
                   first = s_rows[buf].first[warp * R >> 5] >> shift,
                   last = s_rows[buf].last[warp * R >> 5] >> shift;

    // e and b of each row, and the pair of all of them
    float e[N], b[N];
    {
      float xf[N], m[N], gi[N], gr[N];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        xr[j].get(xf + j * V), ir[j].get(gi + j * V), rr[j].get(gr + j * V);
      }
#pragma unroll
      for (int k = 0; k < N; k += 2) {
        sigmoid2<T>(gi + k, gi + k);
        sigmoid2<T>(gr + k, gr + k);
        if (fast) decay2<T, true>(gr + k, ac[0], ac[V - 1], e + k, m + k);
        else decay2<T, false>(gr + k, ac[0], ac[V - 1], e + k, m + k);
        mul2(b[k], b[k + 1], m[k], m[k + 1], gi[k], gi[k + 1]);
        mul2(b[k], b[k + 1], b[k], b[k + 1], xf[k], xf[k + 1]);
      }
    }
    float2 s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = make_float2(1.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!(in >> j & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v) e[j * V + v] = 1.0f, b[j * V + v] = 0.0f;
      }
      if (first >> j & 1) {
        float h0[V];
        if (start_state<V>(p, s_rows[buf].seq[warp * R + j], c, cols, h0)) {
#pragma unroll
          for (int v = 0; v < V; ++v) b[j * V + v] = fmaf(e[j * V + v], h0[v], b[j * V + v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = make_float2(kCut, b[j * V + v]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = compose(s[v], make_float2(e[j * V + v], b[j * V + v]));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_warp[warp][lane * V + v] = s[v];
    __syncthreads();

    // the tile's pair, to every CTA of the cluster
    {
      const int ch = threadIdx.x % C;
      float2 t = s_warp[0][ch];
#pragma unroll
      for (int w = 1; w < W; ++w) t = compose(t, s_warp[w][ch]);
      for (uint32_t k = threadIdx.x / C; k < size; k += blockDim.x / C)
        put_peer(&s_peer[buf][rank][ch], k, t);
    }
    cluster_arrive();
    if (turn + 1 < turns) fetch(tile + size);
    cluster_wait();

    // the state before this warp's rows
    float h[V];
    for (uint32_t k = 0; k < size; ++k) {
      if (k == rank) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = carry[v];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = through(s_peer[buf][k][lane * V + v], carry[v]);
    }
    if (p.saved && warp == 0 && tile * kTile >= lo && tile * kTile < hi) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < cols) p.saved[tile * p.width + c + v] = h[v];
    }
#pragma unroll
    for (int w = 0; w < W - 1; ++w) {
      if (w < warp) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = through(s_warp[w][lane * V + v], h[v]);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool cut = first >> j & 1;
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = cut ? b[j * V + v] : fmaf(e[j * V + v], h[v], b[j * V + v]);
      const int64_t r = tile * kTile + warp * R + j;
      if (p.out && (in >> j & 1) && cols == V) Raw<T, V>::put(out + r * p.os, h);
      if (p.keep_state && (last >> j & 1)) {
        const int64_t slot = seq_slot(p.q, s_rows[buf].seq[warp * R + j]);
        if (slot >= 0 && cols == V) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.state[slot * p.slot_stride + c + v] = h[v];
        }
      }
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
template <typename T, int V>
__global__ void __launch_bounds__(512, 1) k_recur_backward(const Params p) {
  constexpr int W = 16, R = kTile / W, N = R * V, C = 32 * V;
  __shared__ float2 s_down[W][C];  // pairs of states
  __shared__ float2 s_up[W][C];    // pairs of gradients
  __shared__ float2 s_peer[2][kMaxCluster][C];
  __shared__ TileRows s_rows[2];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * V;
  const int cols = c >= p.width ? 0 : static_cast<int>(p.width - c < V ? p.width - c : V);
  float ac[V];
  bool fast = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    ac[v] = v < cols ? __ldg(p.a + c + v) : 0.0f;
    fast = fast && ac[v] > kSeries;
  }
  fast = __all_sync(0xffffffffu, fast);
  const int64_t lo = segment_begin(p, blockIdx.z), hi = segment_begin(p, blockIdx.z + 1);
  const int64_t tile0 = lo / kTile, tiles = hi > lo ? (hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (tiles + size - 1) / size;
  const int64_t top = tile0 + tiles - 1;  // the last tile

  const T* x = static_cast<const T*>(p.x) + c;
  const T* ig = static_cast<const T*>(p.ig) + c;
  const T* rg = static_cast<const T*>(p.rg) + c;
  const T* dout = static_cast<const T*>(p.dout) + c;
  Raw<T, V> xr[R], ir[R], rr[R], gr[R];
  float hs[V] = {};  // the state before the tile, as it was kept
  auto fetch = [&](int64_t tile) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t r = tile * kTile + warp * R + j;
      if (cols == V && r >= lo && r < hi) {
        xr[j].load(x + r * p.xs);
        ir[j].load(ig + r * p.is);
        rr[j].load(rg + r * p.rs);
        gr[j].load(dout + r * p.gs);
      } else {
        xr[j].clear(), ir[j].clear(), rr[j].clear(), gr[j].clear();
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      hs[v] = tile * kTile >= lo && v < cols ? __ldg(p.saved + tile * p.width + c + v) : 0.0f;
    if (threadIdx.x < kTile) place_rows(p.q, tile, lo, hi, &s_rows[(top - tile) / size & 1]);
  };

  float carry[V] = {}, da[V] = {};
  cluster_arrive();  // (every CTA has begun before another one writes to it)
  if (turns > 0) fetch(top - rank);
  cluster_wait();
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t tile = top - (turn * size + rank);
    const int buf = turn & 1;
    __syncthreads();
    const int shift = warp * R & 31;
    const uint32_t in = s_rows[buf].in[warp * R >> 5] >> shift,
                   first = s_rows[buf].first[warp * R >> 5] >> shift,
                   last = s_rows[buf].last[warp * R >> 5] >> shift;

    float e[N], m[N], si[N], sr[N], xf[N], g[N];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      xr[j].get(xf + j * V), ir[j].get(si + j * V), rr[j].get(sr + j * V);
      gr[j].get(g + j * V);
    }
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      sigmoid2<T>(si + k, si + k);
      sigmoid2<T>(sr + k, sr + k);
      if (fast) decay2<T, true>(sr + k, ac[0], ac[V - 1], e + k, m + k);
      else decay2<T, false>(sr + k, ac[0], ac[V - 1], e + k, m + k);
    }
    float2 down[V], up[V];
#pragma unroll
    for (int v = 0; v < V; ++v) down[v] = up[v] = make_float2(1.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!(in >> j & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          e[j * V + v] = 1.0f, m[j * V + v] = xf[j * V + v] = g[j * V + v] = 0.0f;
      }
      float b[V];
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = m[j * V + v] * si[j * V + v] * xf[j * V + v];
      if (first >> j & 1) {
        float h0[V];
        start_state<V>(p, s_rows[buf].seq[warp * R + j], c, cols, h0);
#pragma unroll
        for (int v = 0; v < V; ++v)
          down[v] = make_float2(kCut, fmaf(e[j * V + v], h0[v], b[v]));
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) down[v] = compose(down[v], make_float2(e[j * V + v], b[v]));
      }
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      if (last >> j & 1) {
        if (p.dstate) {
          const float* d = p.dstate + s_rows[buf].seq[warp * R + j] * p.width + c;
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v < cols) g[j * V + v] += __ldg(d + v);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) up[v] = make_float2(kCut, e[j * V + v] * g[j * V + v]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          up[v] = compose(up[v], make_float2(e[j * V + v], e[j * V + v] * g[j * V + v]));
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s_down[warp][lane * V + v] = down[v];
      s_up[warp][lane * V + v] = up[v];
    }
    __syncthreads();
    {
      const int ch = threadIdx.x % C;
      float2 t = s_up[W - 1][ch];
#pragma unroll
      for (int w = W - 2; w >= 0; --w) t = compose(t, s_up[w][ch]);
      for (uint32_t k = threadIdx.x / C; k < size; k += blockDim.x / C)
        put_peer(&s_peer[buf][rank][ch], k, t);
    }
    cluster_arrive();
    // the states before each row, meanwhile
    float h[V], hp[N];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = hs[v];
    for (int w = 0; w < warp; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = through(s_down[w][lane * V + v], h[v]);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (first >> j & 1) start_state<V>(p, s_rows[buf].seq[warp * R + j], c, cols, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = j * V + v;
        hp[k] = h[v];
        h[v] = fmaf(e[k], h[v], m[k] * si[k] * xf[k]);
      }
    }
    if (turn + 1 < turns) fetch(tile - size);
    cluster_wait();

    // the gradient that comes to this warp's last row from the rows behind it
    float gc[V];
    for (uint32_t k = 0; k < size; ++k) {
      if (k == rank) {
#pragma unroll
        for (int v = 0; v < V; ++v) gc[v] = carry[v];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) carry[v] = through(s_peer[buf][k][lane * V + v], carry[v]);
    }
    for (int w = W - 1; w > warp; --w) {
#pragma unroll
      for (int v = 0; v < V; ++v) gc[v] = through(s_up[w][lane * V + v], gc[v]);
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const bool cut = last >> j & 1;
      float dx[V], di[V], dr[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = j * V + v;
        const float gk = cut ? g[k] : g[k] + gc[v];
        const float over = m[k] > 0.0f ? (Elem<T>::kExactSilu ? sr[k] / m[k]
                                                              : sr[k] * rcp_approx(m[k]))
                                       : 0.0f;
        dx[v] = gk * m[k] * si[k];
        di[v] = dx[v] * xf[k] * (1.0f - si[k]);
        const float dpr = gk * (hp[k] * e[k] * sr[k] - si[k] * xf[k] * e[k] * e[k] * over);
        dr[v] = dpr * ac[v] * (1.0f - sr[k]);
        if (in >> j & 1) da[v] += dpr;
        gc[v] = e[k] * gk;
      }
      const int64_t r = tile * kTile + warp * R + j;
      if (r >= lo && r < hi && cols == V) {
        if (!(in >> j & 1)) {  // a row of no sequence
#pragma unroll
          for (int v = 0; v < V; ++v) dx[v] = di[v] = dr[v] = 0.0f;
        }
        Raw<T, V>::put(static_cast<T*>(p.dx) + r * p.dxs + c, dx);
        Raw<T, V>::put(static_cast<T*>(p.dig) + r * p.dis + c, di);
        Raw<T, V>::put(static_cast<T*>(p.drg) + r * p.drs + c, dr);
      }
      if (p.dinitial && (first >> j & 1)) {
        const int64_t s = s_rows[buf].seq[warp * R + j];
        const bool resumes = seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v < cols) p.dinitial[s * p.width + c + v] = resumes ? gc[v] : 0.0f;
      }
    }
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
#pragma unroll
  for (int v = 0; v < V; ++v) s_up[warp][lane * V + v].x = da[v];
  __syncthreads();
  if (threadIdx.x < C) {
    float t = 0.0f;
    for (int w = 0; w < W; ++w) t += s_up[w][threadIdx.x].x;
    put_peer(&s_peer[turns & 1][rank][threadIdx.x], 0, make_float2(t, 0.0f));
  }
  cluster_arrive();
  cluster_wait();
  const int64_t ch = static_cast<int64_t>(blockIdx.y) * C + threadIdx.x;
  if (rank == 0 && threadIdx.x < C && ch < p.width) {
    float t = 0.0f;
    for (uint32_t k = 0; k < size; ++k) t += s_peer[turns & 1][k][threadIdx.x].x;
    p.da[blockIdx.z * p.width + ch] = t;
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

template <typename K>
int launch_cluster(K kernel, const Params& p, int64_t blocks, Split s, unsigned threads,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.cluster), static_cast<unsigned>(blocks),
                     static_cast<unsigned>(s.segments));
  cfg.blockDim = dim3(threads);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  return GGRN_OK;
}

int64_t blocks_of(int64_t width, int v) { return (width + 32 * v - 1) / (32 * v); }

template <typename T, int V>
int launch_forward(Params& p, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width, V);
  const Split k = split_rows(p.q.rows, p.q.seqs, blocks, sizeof(T) == 2 ? 3 : 2);
  p.segments = k.segments;
  return launch_cluster(k_recur<T, V>, p, blocks, k, 256, s);
}
template <typename T, int V>
int launch_backward(Params& p, float* sums, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width, V);
  const Split k = split_rows(p.q.rows, p.q.seqs, blocks, 1);
  p.segments = k.segments;
  float* const da = p.da;
  if (k.segments > 1) p.da = sums;
  const int st = launch_cluster(k_recur_backward<T, V>, p, blocks, k, 512, s);
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

// Widths that a grid's second axis holds with one channel a lane.
constexpr int64_t kMostColumns = int64_t{65535} * 32;

struct Matrix {
  const void* p;
  int64_t stride;
};
// Pairs of channels: every row of every matrix starts on one.
bool pairs(int64_t rows, int64_t width, int es, std::initializer_list<Matrix> ms) {
  if (width % 2) return false;
  for (const Matrix& m : ms)
    if (!mixer::aligned_to(m.p, 2 * es) || (rows > 1 && m.stride % 2)) return false;
  return true;
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
  const bool two = pairs(c.rows, c.width, es, {{c.x, p.xs}, {c.input_gate, p.is},
                                               {c.decay_gate, p.rs}, {c.out, p.os}});
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step) {
    if (c.dtype == kF32) return two ? launch_step<float, 2>(p, s) : launch_step<float, 1>(p, s);
    if (c.dtype == kF16) return two ? launch_step<__half, 2>(p, s) : launch_step<__half, 1>(p, s);
    return two ? launch_step<__nv_bfloat16, 2>(p, s) : launch_step<__nv_bfloat16, 1>(p, s);
  }
  if (c.dtype == kF32) return two ? launch_forward<float, 2>(p, s) : launch_forward<float, 1>(p, s);
  if (c.dtype == kF16)
    return two ? launch_forward<__half, 2>(p, s) : launch_forward<__half, 1>(p, s);
  return two ? launch_forward<__nv_bfloat16, 2>(p, s) : launch_forward<__nv_bfloat16, 1>(p, s);
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
  // the most segments that split_rows makes, by pairs of channels or one by one
  int64_t most = 1;
  for (int v = 1; v <= 2; ++v) {
    const int64_t n = split_rows(c.rows, c.seqs, blocks_of(c.width, v), 1).segments;
    if (n > most) most = n;
  }
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

template <typename T, int V>
int backward(Params& p, const Space& need, void* workspace, cudaStream_t s) {
  if (!p.saved && p.q.rows > 0) {
    Params f = p;
    p.saved = f.saved = static_cast<float*>(workspace);
    const int st = launch_forward<T, V>(f, s);
    if (st != GGRN_OK) return st;
  }
  float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + need.saved);
  return launch_backward<T, V>(p, sums, s);
}

int run_backward(const ggrn_recur_backward_call* call, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_recur_backward_call& c = *call;
  Params p = {};
  const int st = check_backward(c, &p);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  const bool two = pairs(c.rows, c.width, es,
                         {{c.dout, p.gs}, {c.x, p.xs}, {c.input_gate, p.is}, {c.decay_gate, p.rs},
                          {c.dx, p.dxs}, {c.dinput_gate, p.dis}, {c.ddecay_gate, p.drs}});
  const Space need = space_of(c);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* const w = c.workspace;
  if (c.dtype == kF32)
    return two ? backward<float, 2>(p, need, w, s) : backward<float, 1>(p, need, w, s);
  if (c.dtype == kF16)
    return two ? backward<__half, 2>(p, need, w, s) : backward<__half, 1>(p, need, w, s);
  return two ? backward<__nv_bfloat16, 2>(p, need, w, s)
             : backward<__nv_bfloat16, 1>(p, need, w, s);
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
