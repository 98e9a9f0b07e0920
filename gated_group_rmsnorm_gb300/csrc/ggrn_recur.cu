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
  int mute;            // self-test: nothing is sent, so that the waits run out
  unsigned int* fault; // device status word
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
// exp(p) - 1 = p + p^2 (..) where p > -1/4, with a polynomial through the
// Chebyshev points of that range (within 2^-26 of it), and e = 1 + that, m^2 =
// 1 - e^2 = -(e - 1)(2 + (e - 1)): neither loses digits to cancellation where
// decays are slow (an exponential that is off by an ulp to one side next to 1 is
// off by a thousand after a thousand rows), and slow channels take no second
// exponential.  FAST: no decay of the warp's channels is below exp(-1/4).
// (Constants stand in scalar instructions, which hold them; pairs would need
// them in registers.)
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
#pragma unroll
    for (int k = 0; k < 2; ++k) s[k] = rcp_approx(1.0f + ex2_approx(z[k] * -1.4426950408889634f));
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
  float s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float c = fmaf(7.67176877707243e-3f, p[k], 4.1564859449863434e-2f);
    c = fmaf(c, p[k], 1.666616052389145e-1f);
    c = fmaf(c, p[k], 4.999999701976776e-1f);
    c = fmaf(c, p[k], 1.0f);
    s[k] = c * p[k];  // e - 1
    e[k] = 1.0f + s[k];
  }
  if constexpr (!FAST) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (!(p[k] > kSeries)) beyond_series<T>(p[k], e[k], s[k]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float q = -s[k] * (2.0f + s[k]);
    m[k] = Elem<T>::kExactSilu ? sqrtf(q) : sqrt_approx(q);
  }
}

// ---------------------------------------------------------------------------
// Clusters.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void all_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void all_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Stores v at the place of *mine in the shared memory of CTA `rank`.
__device__ __forceinline__ void put_peer(const float4* mine, uint32_t rank, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                   map_to_rank(smem_u32(mine), rank)),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// What the CTAs of a cluster send each other every turn: a pair for each lane and
// whether it is cut, by asynchronous remote stores that count their bytes on a
// barrier of the CTA they go to, so that no turn waits for a CTA's other memory
// operations.  Two turns' places: a CTA sends those of turn t + 2 when it has those
// of turn t + 1, which the others send when they are through with turn t.
//
// Waits are bounded: one that runs out (about a second) sets `failed`, after which
// the CTA's waits return at once and its outputs have no meaning; the status word
// says so.  The CTAs of a cluster end together, so that nothing is sent to one that
// has ended.
constexpr uint32_t kFaultRecurWait = 128u;
constexpr long long kWaitClocks = 2000000000ll;
struct Mail {
  float4 pair[2][kMaxCluster][32];
  int cut[2][kMaxCluster];
  unsigned long long landed[2];
  volatile uint32_t failed;
};
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ void wait_poll(uint32_t bar, uint32_t parity, volatile uint32_t* failed) {
  const long long start = clock64();
  do {
    if (*failed || try_phase(bar, parity)) return;
  } while (clock64() - start < kWaitClocks);
  *failed = 1;
}
// Before the arrival of every CTA of the cluster that comes before its first mail.
__device__ __forceinline__ void mail_init(Mail& m) {
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&m.landed[0]), 1);
    mbar_init(smem_u32(&m.landed[1]), 1);
    m.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
}
// A whole warp sends to CTA `to`.
__device__ __forceinline__ void mail_send(Mail& m, int buf, int rank, int to, const float4& v,
                                          bool cut) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar = map_to_rank(smem_u32(&m.landed[buf]), to);
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
      ::"r"(map_to_rank(smem_u32(&m.pair[buf][rank][lane]), to)),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
      : "memory");
  if (lane == 0)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                     map_to_rank(smem_u32(&m.cut[buf][rank]), to)),
                 "r"(cut ? 1u : 0u), "r"(bar)
                 : "memory");
}
// One thread, before the wait: how much will land.
__device__ __forceinline__ void mail_expect(Mail& m, int buf, int size) {
  mbar_expect_tx(smem_u32(&m.landed[buf]), static_cast<uint32_t>(size) * (32 * 16 + 4));
}
__device__ __forceinline__ void mail_wait(Mail& m, int buf, uint32_t parity) {
  const uint32_t bar = smem_u32(&m.landed[buf]);
  if (!try_phase(bar, parity)) wait_poll(bar, parity, &m.failed);
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
// outside [lo, hi) and channels behind the last one become zeros.  `whole`: there
// are none of either.
template <typename T, int THREADS>
__device__ __forceinline__ void copy_tile(T* to, const void* base, int64_t stride, int64_t c0,
                                          int64_t width, int64_t tile, int64_t lo, int64_t hi,
                                          int chunk, bool whole) {
  constexpr int ES = sizeof(T);
  const T* from = static_cast<const T*>(base) + c0;
  const int64_t r0 = tile * kTile;
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  constexpr int E = 16 / ES, ROW = kCols / E, ROWS = THREADS / ROW;  // 16-byte chunks
  if (chunk == 16 && whole) {
    const T* p = from + (r0 + threadIdx.x / ROW) * stride + threadIdx.x % ROW * E;
    const int64_t step = ROWS * stride;
#pragma unroll
    for (int k = 0; k < kTile / ROWS; ++k, p += step)
      copy_async<16>(at + (threadIdx.x + k * THREADS) * 16, p, 16);
    return;
  }
  const int cols = static_cast<int>(width - c0 < kCols ? width - c0 : kCols);
  if (chunk == 16) {
#pragma unroll 1
    for (int k = threadIdx.x; k < kTile * ROW; k += THREADS) {
      const int row = k / ROW, c = k % ROW * E;
      const bool ok = r0 + row >= lo && r0 + row < hi && c < cols;
      copy_async<16>(at + k * 16, ok ? from + (r0 + row) * stride + c : from, ok ? 16 : 0);
    }
  } else if (chunk == 4) {
    constexpr int E4 = 4 / ES, ROW4 = kCols / E4;
#pragma unroll 2
    for (int k = threadIdx.x; k < kTile * ROW4; k += THREADS) {
      const int row = k / ROW4, c = k % ROW4 * E4;
      const bool ok = r0 + row >= lo && r0 + row < hi && c < cols;
      copy_async<4>(at + k * 4, ok ? from + (r0 + row) * stride + c : from,
                    !ok ? 0 : cols - c < E4 ? ES : 4);
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

// What a CTA knows for all of its tiles.
struct Place {
  int64_t lo, hi;   // rows of its segment
  int64_t c0, c;    // first channel of the CTA and of the lane
  int cols;         // the lane's channels (0 to 2)
  int rank, size;   // in its cluster
  float ac[2];
};
__device__ __forceinline__ Place find_place(const Params& p) {
  Place w;
  const int lane = threadIdx.x & 31;
  w.rank = static_cast<int>(cluster_ctarank());
  w.size = static_cast<int>(cluster_size());
  w.c0 = static_cast<int64_t>(blockIdx.y) * kCols;
  w.c = w.c0 + lane * 2;
  w.cols = w.c >= p.width ? 0 : p.width - w.c < 2 ? 1 : 2;
  w.lo = segment_begin(p, blockIdx.z);
  w.hi = segment_begin(p, blockIdx.z + 1);
#pragma unroll
  for (int v = 0; v < 2; ++v) w.ac[v] = v < w.cols ? __ldg(p.a + w.c + v) : 0.0f;
  return w;
}
__device__ __forceinline__ bool whole_tile(const Params& p, const Place& w, int64_t tile) {
  return tile * kTile >= w.lo && (tile + 1) * kTile <= w.hi && w.c0 + kCols <= p.width;
}

// ---------------------------------------------------------------------------
// Prompts.  Four warps of sixteen rows each: an element costs about 25
// instructions of its own, what a tile costs besides is shared by 32 elements of
// a thread.
// ---------------------------------------------------------------------------
namespace forward {

constexpr int W = 4, R = kTile / W, kThreads = 32 * W;

struct Shared {
  float4 pair[W][32];
  Mail mail;
  TileRows rows;
};

template <typename T>
__device__ __forceinline__ void fetch(const Params& p, const Place& w, T* to, int64_t tile) {
  const bool whole = whole_tile(p, w, tile);
  const auto copy = [&](int k, const void* base, int64_t stride) {
    copy_tile<T, kThreads>(to + k * kTile * kCols, base, stride, w.c0, p.width, tile, w.lo, w.hi,
                           p.chunk, whole);
  };
  copy(0, p.x, p.xs), copy(1, p.ig, p.is), copy(2, p.rg, p.rs);
}

// One tile.  INSIDE: all of its rows are those of one sequence, neither its first
// nor its last.  FAST: see decay2.  Takes the state before the cluster's tiles and
// gives the one behind them.
template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ float2 turn_of(const Params& p, const Place& w, Shared& sh, T* tiles,
                                          int64_t tile, int64_t next, int64_t turn, float2 state) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int buf = turn & 1;
  const uint32_t parity = turn >> 1 & 1;
  const T* mine = tiles + warp * R * kCols + lane * 2;
  const TileRows& t = sh.rows;
  // e and b of the warp's rows, and the pair of all of them
  float e[R][2], b[R][2];
  float4 s = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float x[2], gi[2], gr[2], m[2];
    get2(mine + j * kCols, x);
    get2(mine + (kTile + j) * kCols, gi);
    get2(mine + (2 * kTile + j) * kCols, gr);
    sigmoid2<T>(gi, gi);
    sigmoid2<T>(gr, gr);
    decay2<T, FAST>(gr, w.ac[0], w.ac[1], e[j], m);
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
        if (start_state<2>(p, t.seq[row], w.c, w.cols, h))
          fma2(b[j][0], b[j][1], e[j][0], e[j][1], h[0], h[1], b[j][0], b[j][1]);
        e[j][0] = e[j][1] = kCut;
      }
    }
    compose<!INSIDE>(s, make_float4(e[j][0], e[j][1], b[j][0], b[j][1]));
  }
  sh.pair[warp][lane] = s;
  const bool cut = !INSIDE && (t.first[0] | t.first[1]) != 0;
  __syncthreads();
  if (next >= 0) fetch(p, w, tiles, next);

  // the pair of the rows before this warp's in the tile, and of the whole tile
  float4 before = make_float4(1.0f, 1.0f, 0.0f, 0.0f), whole = sh.pair[0][lane];
#pragma unroll
  for (int k = 1; k < W; ++k) {
    if (k == warp) before = whole;
    compose<!INSIDE>(whole, sh.pair[k][lane]);
  }
  float carry[2] = {state.x, state.y}, h[2] = {state.x, state.y};
  if (w.size > 1) {
    if (threadIdx.x == 0) mail_expect(sh.mail, buf, w.size);
    if (!p.mute)
      for (int k = warp; k < w.size; k += W) mail_send(sh.mail, buf, w.rank, k, whole, cut);
    mail_wait(sh.mail, buf, parity);
    bool cuts = false;
    for (int k = 0; k < w.size; ++k) cuts = cuts || sh.mail.cut[buf][k] != 0;
    if (cuts) {
      for (int k = 0; k < w.size; ++k) {
        if (k == w.rank) h[0] = carry[0], h[1] = carry[1];
        through<true>(sh.mail.pair[buf][k][lane], carry);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= w.size) break;
        if (k == w.rank) h[0] = carry[0], h[1] = carry[1];
        through<false>(sh.mail.pair[buf][k][lane], carry);
      }
    }
  } else {
    through<!INSIDE>(whole, carry);
  }
  if (p.saved && warp == 0 && tile * kTile >= w.lo && tile * kTile < w.hi) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (v < w.cols) p.saved[tile * p.width + w.c + v] = h[v];
  }
  through<!INSIDE>(before, h);
  if constexpr (INSIDE) {
    if (p.out) {
      T* at = static_cast<T*>(p.out) + (tile * kTile + warp * R) * p.os + w.c;
      if (p.pairs && w.cols == 2) {
#pragma unroll
        for (int j = 0; j < R; ++j, at += p.os) {
          fma2(h[0], h[1], e[j][0], e[j][1], h[0], h[1], b[j][0], b[j][1]);
          Raw<T, 2>::put(at, h);
        }
      } else {
#pragma unroll
        for (int j = 0; j < R; ++j, at += p.os) {
          fma2(h[0], h[1], e[j][0], e[j][1], h[0], h[1], b[j][0], b[j][1]);
          put2<T>(at, 0, h, w.cols, false);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      through<true>(make_float4(e[j][0], e[j][1], b[j][0], b[j][1]), h);
      const int row = warp * R + j;
      if (p.out && (t.in[row >> 5] >> (row & 31) & 1))
        put2<T>(p.out, (tile * kTile + row) * p.os + w.c, h, w.cols, p.pairs);
      if (p.keep_state && (t.last[row >> 5] >> (row & 31) & 1)) {
        const int64_t slot = seq_slot(p.q, t.seq[row]);
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (slot >= 0 && v < w.cols) p.state[slot * p.slot_stride + w.c + v] = h[v];
      }
    }
    __syncthreads();  // (the next turn's search writes rows)
  }
  return make_float2(carry[0], carry[1]);
}
// The forms that few tiles take, out of the way of the loop's instructions and
// registers.
template <typename T, bool INSIDE, bool FAST>
__device__ __noinline__ float2 turn_apart(const Params& p, Place w, Shared& sh, T* tiles,
                                          int64_t tile, int64_t next, int64_t turn, float2 state) {
  return turn_of<T, INSIDE, FAST>(p, w, sh, tiles, tile, next, turn, state);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    k_recur(const __grid_constant__ Params p) {
  extern __shared__ uint4 s_tile[];
  __shared__ Shared sh;
  T* const tiles = reinterpret_cast<T*>(s_tile);  // x, input gate, decay gate
  pdl_wait();
  pdl_launch_dependents();
  mail_init(sh.mail);
  all_arrive();  // (every CTA has begun before another one writes to it)
  const Place w = find_place(p);
  const int64_t tile0 = w.lo / kTile, count = w.hi > w.lo ? (w.hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (count + w.size - 1) / w.size;
  int64_t tile = tile0 + w.rank;
  if (turns > 0) fetch(p, w, tiles, tile);
  const bool fast = __all_sync(0xffffffffu, w.ac[0] > kSeries && w.ac[1] > kSeries);
  all_wait();

  float2 state = make_float2(0.0f, 0.0f);  // before the cluster's tiles
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn, tile += w.size) {
    const int64_t next = turn + 1 < turns ? tile + w.size : -1;
    const bool inside = known.inside(tile) && (tile + 1) * kTile <= w.hi;
    if (!inside && threadIdx.x < kTile) place_rows(p.q, tile, w.lo, w.hi, &sh.rows);
    copies_wait();
    __syncthreads();
    if (inside && fast) {
      state = turn_of<T, true, true>(p, w, sh, tiles, tile, next, turn, state);
    } else if (inside) {
      state = turn_apart<T, true, false>(p, w, sh, tiles, tile, next, turn, state);
    } else {
      known.begin = sh.rows.begin, known.end = sh.rows.end;
      state = turn_apart<T, false, false>(p, w, sh, tiles, tile, next, turn, state);
    }
  }
  if (p.keep_state && threadIdx.x < 32) {
    each_empty(p.q, static_cast<int64_t>(blockIdx.z) * w.size + w.rank,
               static_cast<int64_t>(w.size) * p.segments, [&](int64_t s) {
                 const int64_t slot = seq_slot(p.q, s);
                 if (slot < 0 || seq_resumes(p.q, s)) return;
                 for (int v = 0; v < w.cols; ++v) p.state[slot * p.slot_stride + w.c + v] = 0.0f;
               });
  }
  if (w.size > 1) {
    if (threadIdx.x == 0 && sh.mail.failed) atomicOr(p.fault, kFaultRecurWait);
    all_arrive();
    all_wait();
  }
}

}  // namespace forward

// ---------------------------------------------------------------------------
// Gradients.  Eight warps of eight rows each; the cluster's tiles go from the
// last rows to the first, rank 0 has the last of them.
// ---------------------------------------------------------------------------
namespace backward {

constexpr int W = 8, R = kTile / W, kThreads = 32 * W;
static_assert(W >= kMaxCluster, "a warp to each CTA that the tile's pair goes to");
constexpr int kInput = kTile * kCols;  // elements of an input's tile

struct Shared {
  float4 down[W][32];  // pairs of states
  float4 up[W][32];    // pairs of gradients
  Mail mail;
  TileRows rows;
};

// Tiles of the inputs in shared memory: two of 16-bit types, one of f32.
template <typename T>
constexpr int stages() {
  return sizeof(T) == 2 ? 2 : 1;
}

template <typename T>
__device__ __forceinline__ void fetch(const Params& p, const Place& w, T* to, int64_t tile) {
  const bool whole = whole_tile(p, w, tile);
  const auto copy = [&](int k, const void* base, int64_t stride) {
    copy_tile<T, kThreads>(to + k * kInput, base, stride, w.c0, p.width, tile, w.lo, w.hi, p.chunk,
                           whole);
  };
  copy(0, p.x, p.xs), copy(1, p.ig, p.is), copy(2, p.rg, p.rs), copy(3, p.dout, p.gs);
}

struct Carry {
  float g[2];   // the gradient of the state behind the cluster's tiles
  float da[2];
};

template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ Carry turn_of(const Params& p, const Place& w, Shared& sh, T* ring,
                                         int64_t tile, int64_t next, int64_t turn, Carry carry) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int buf = turn & 1;
  const uint32_t parity = turn >> 1 & 1;
  T* const tiles = ring + (stages<T>() == 2 ? buf : 0) * 4 * kInput;
  const T* mine = tiles + warp * R * kCols + lane * 2;
  const TileRows& t = sh.rows;
  float h[2];  // the state before the tile, as it was kept
#pragma unroll
  for (int v = 0; v < 2; ++v)
    h[v] = tile * kTile >= w.lo && v < w.cols ? __ldg(p.saved + tile * p.width + w.c + v) : 0.0f;
  if (stages<T>() == 2 && next != INT64_MIN) fetch(p, w, ring + (buf ^ 1) * 4 * kInput, next);
  const uint32_t in = INSIDE ? ~0u : t.in[warp * R >> 5] >> (warp * R & 31),
                 first = INSIDE ? 0u : t.first[warp * R >> 5] >> (warp * R & 31),
                 last = INSIDE ? 0u : t.last[warp * R >> 5] >> (warp * R & 31);

  float e[R][2], m[R][2], si[R][2], sr[R][2], b[R][2];
  float4 down = make_float4(1.0f, 1.0f, 0.0f, 0.0f), up = down;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float x[2];
    get2(mine + j * kCols, x);
    get2(mine + kInput + j * kCols, si[j]);
    get2(mine + 2 * kInput + j * kCols, sr[j]);
    sigmoid2<T>(si[j], si[j]);
    sigmoid2<T>(sr[j], sr[j]);
    decay2<T, FAST>(sr[j], w.ac[0], w.ac[1], e[j], m[j]);
    mul2(b[j][0], b[j][1], m[j][0], m[j][1], si[j][0], si[j][1]);
    mul2(b[j][0], b[j][1], b[j][0], b[j][1], x[0], x[1]);
    if (!INSIDE && !(in >> j & 1)) {
      e[j][0] = e[j][1] = 1.0f;
      b[j][0] = b[j][1] = 0.0f;
    }
    if (!INSIDE && (first >> j & 1)) {
      float h0[2];
      start_state<2>(p, t.seq[warp * R + j], w.c, w.cols, h0);
      fma2(h0[0], h0[1], e[j][0], e[j][1], h0[0], h0[1], b[j][0], b[j][1]);
      down = make_float4(kCut, kCut, h0[0], h0[1]);
    } else {
      compose<!INSIDE>(down, make_float4(e[j][0], e[j][1], b[j][0], b[j][1]));
    }
  }
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    float g[2];
    get2(mine + 3 * kInput + j * kCols, g);
    if (!INSIDE && !(in >> j & 1)) continue;
    const bool end = !INSIDE && (last >> j & 1);
    if (end) end_gradient(p, t.seq[warp * R + j], w.c, w.cols, g);
    mul2(g[0], g[1], g[0], g[1], e[j][0], e[j][1]);
    if (end) up = make_float4(kCut, kCut, g[0], g[1]);
    else compose<!INSIDE>(up, make_float4(e[j][0], e[j][1], g[0], g[1]));
  }
  sh.down[warp][lane] = down;
  sh.up[warp][lane] = up;
  const bool cut = !INSIDE && (t.last[0] | t.last[1]) != 0;
  __syncthreads();
  // the pair of the rows behind this warp's in the tile, and of the whole tile
  float4 behind = make_float4(1.0f, 1.0f, 0.0f, 0.0f), whole = sh.up[W - 1][lane];
#pragma unroll
  for (int k = W - 2; k >= 0; --k) {
    if (k == warp) behind = whole;
    compose<!INSIDE>(whole, sh.up[k][lane]);
  }
  if (w.size > 1) {
    if (threadIdx.x == 0) mail_expect(sh.mail, buf, w.size);
    if (warp < w.size) mail_send(sh.mail, buf, w.rank, warp, whole, cut);
  }
  // the states before each row, meanwhile
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    if (k < warp) through<!INSIDE>(sh.down[k][lane], h);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (!INSIDE && (first >> j & 1)) start_state<2>(p, t.seq[warp * R + j], w.c, w.cols, h);
    const float b0 = b[j][0], b1 = b[j][1];
    b[j][0] = h[0], b[j][1] = h[1];  // (from here on the state before the row)
    if (INSIDE || (in >> j & 1)) fma2(h[0], h[1], e[j][0], e[j][1], h[0], h[1], b0, b1);
  }
  // the gradient that comes to this warp's last row from the rows behind it
  float gc[2] = {carry.g[0], carry.g[1]};
  if (w.size > 1) {
    mail_wait(sh.mail, buf, parity);
    bool cuts = false;
    for (int k = 0; k < w.size; ++k) cuts = cuts || sh.mail.cut[buf][k] != 0;
    if (cuts) {
      for (int k = 0; k < w.size; ++k) {
        if (k == w.rank) gc[0] = carry.g[0], gc[1] = carry.g[1];
        through<true>(sh.mail.pair[buf][k][lane], carry.g);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= w.size) break;
        if (k == w.rank) gc[0] = carry.g[0], gc[1] = carry.g[1];
        through<false>(sh.mail.pair[buf][k][lane], carry.g);
      }
    }
  } else {
    through<!INSIDE>(whole, carry.g);
  }
  through<!INSIDE>(behind, gc);

  const int64_t row0 = tile * kTile + warp * R;
  T* dx_at = static_cast<T*>(p.dx) + row0 * p.dxs + w.c;
  T* di_at = static_cast<T*>(p.dig) + row0 * p.dis + w.c;
  T* dr_at = static_cast<T*>(p.drg) + row0 * p.drs + w.c;
  const bool pairs = p.pairs && w.cols == 2;
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    float g[2], x[2], dx[2], di[2], dr[2], t1[2], t2[2];
    get2(mine + j * kCols, x);
    get2(mine + 3 * kInput + j * kCols, g);
    if (!INSIDE && (last >> j & 1)) end_gradient(p, t.seq[warp * R + j], w.c, w.cols, g);
    else g[0] += gc[0], g[1] += gc[1];
    // dx = g m i,  di = dx x (1 - i)
    mul2(dx[0], dx[1], m[j][0], m[j][1], si[j][0], si[j][1]);
    mul2(dx[0], dx[1], dx[0], dx[1], g[0], g[1]);
    mul2(di[0], di[1], dx[0], dx[1], x[0], x[1]);
    mul2(di[0], di[1], di[0], di[1], 1.0f - si[j][0], 1.0f - si[j][1]);
    // g e r (h - i x e / m)
    float over[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      over[v] = Elem<T>::kExactSilu ? 1.0f / m[j][v] : rcp_approx(m[j][v]);
      if (!(m[j][v] > 0.0f)) over[v] = 0.0f;
    }
    mul2(t2[0], t2[1], si[j][0], si[j][1], x[0], x[1]);
    mul2(t2[0], t2[1], t2[0], t2[1], -e[j][0], -e[j][1]);
    fma2(t1[0], t1[1], t2[0], t2[1], over[0], over[1], b[j][0], b[j][1]);
    mul2(t2[0], t2[1], e[j][0], e[j][1], sr[j][0], sr[j][1]);
    mul2(t1[0], t1[1], t1[0], t1[1], t2[0], t2[1]);
    mul2(t1[0], t1[1], t1[0], t1[1], g[0], g[1]);
    mul2(dr[0], dr[1], t1[0], t1[1], w.ac[0], w.ac[1]);
    mul2(dr[0], dr[1], dr[0], dr[1], 1.0f - sr[j][0], 1.0f - sr[j][1]);
    if (INSIDE || (in >> j & 1)) {
      carry.da[0] += t1[0], carry.da[1] += t1[1];
      mul2(gc[0], gc[1], e[j][0], e[j][1], g[0], g[1]);
    } else {  // a row of no sequence
#pragma unroll
      for (int v = 0; v < 2; ++v) dx[v] = di[v] = dr[v] = 0.0f;
    }
    if (INSIDE || (row0 + j >= w.lo && row0 + j < w.hi)) {
      if (pairs) {
        Raw<T, 2>::put(dx_at + j * p.dxs, dx);
        Raw<T, 2>::put(di_at + j * p.dis, di);
        Raw<T, 2>::put(dr_at + j * p.drs, dr);
      } else {
        put2<T>(dx_at, j * p.dxs, dx, w.cols, false);
        put2<T>(di_at, j * p.dis, di, w.cols, false);
        put2<T>(dr_at, j * p.drs, dr, w.cols, false);
      }
    }
    if (!INSIDE && p.dinitial && (first >> j & 1)) {
      const int64_t s = t.seq[warp * R + j];
      const bool resumes = seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (v < w.cols) p.dinitial[s * p.width + w.c + v] = resumes ? gc[v] : 0.0f;
    }
  }
  // (the next turn's search writes rows, its copies the tile)
  if (!INSIDE || stages<T>() == 1) __syncthreads();
  if (stages<T>() == 1 && next != INT64_MIN) fetch(p, w, ring, next);
  return carry;
}
template <typename T, bool INSIDE, bool FAST>
__device__ __noinline__ Carry turn_apart(const Params& p, Place w, Shared& sh, T* ring,
                                         int64_t tile, int64_t next, int64_t turn, Carry carry) {
  return turn_of<T, INSIDE, FAST>(p, w, sh, ring, tile, next, turn, carry);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    k_recur_backward(const __grid_constant__ Params p) {
  extern __shared__ uint4 s_tile[];
  __shared__ Shared sh;
  T* const ring = reinterpret_cast<T*>(s_tile);  // x, input gate, decay gate, dout
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  mail_init(sh.mail);
  all_arrive();  // (every CTA has begun before another one writes to it)
  const Place w = find_place(p);
  const int64_t tile0 = w.lo / kTile, count = w.hi > w.lo ? (w.hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (count + w.size - 1) / w.size;
  int64_t tile = tile0 + count - 1 - w.rank;
  if (turns > 0) fetch(p, w, ring, tile);
  const bool fast = __all_sync(0xffffffffu, w.ac[0] > kSeries && w.ac[1] > kSeries);
  all_wait();

  Carry carry = {};
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn, tile -= w.size) {
    const int64_t next = turn + 1 < turns ? tile - w.size : INT64_MIN;
    const bool inside = tile * kTile >= w.lo && known.inside(tile);
    if (!inside && threadIdx.x < kTile) place_rows(p.q, tile, w.lo, w.hi, &sh.rows);
    copies_wait();
    __syncthreads();
    if (inside && fast) {
      carry = turn_of<T, true, true>(p, w, sh, ring, tile, next, turn, carry);
    } else if (inside) {
      carry = turn_apart<T, true, false>(p, w, sh, ring, tile, next, turn, carry);
    } else {
      // (of the tile's first row: the tiles before it come next)
      known.begin = known.end = 0;
      if (tile * kTile >= w.lo && tile * kTile < w.hi)
        seq_range(p.q, sh.rows.seq[0], known.begin, known.end);
      carry = turn_apart<T, false, false>(p, w, sh, ring, tile, next, turn, carry);
    }
  }
  if (p.dinitial && warp == 0) {
    each_empty(p.q, static_cast<int64_t>(blockIdx.z) * w.size + w.rank,
               static_cast<int64_t>(w.size) * p.segments, [&](int64_t s) {
                 const bool keep = p.dstate && seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
                 for (int v = 0; v < w.cols; ++v) {
                   const int64_t k = s * p.width + w.c + v;
                   p.dinitial[k] = keep ? __ldg(p.dstate + k) : 0.0f;
                 }
               });
  }
  // da: the warps' sums, then the CTAs' in rank 0
  __syncthreads();
  sh.up[warp][lane] = make_float4(carry.da[0], carry.da[1], 0.0f, 0.0f);
  __syncthreads();
  if (warp == 0) {
    float4 t = sh.up[0][lane];
    for (int k = 1; k < W; ++k) t.x += sh.up[k][lane].x, t.y += sh.up[k][lane].y;
    put_peer(&sh.mail.pair[turns & 1][w.rank][lane], 0, t);
    if (lane == 0 && sh.mail.failed) atomicOr(p.fault, kFaultRecurWait);
  }
  all_arrive();
  all_wait();
  if (w.rank == 0 && warp == 0) {
    float t[2] = {0.0f, 0.0f};
    for (int k = 0; k < w.size; ++k) {
      t[0] += sh.mail.pair[turns & 1][k][lane].x;
      t[1] += sh.mail.pair[turns & 1][k][lane].y;
    }
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (v < w.cols) p.da[blockIdx.z * p.width + w.c + v] = t[v];
  }
}

}  // namespace backward

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
int launch_cluster(void (*kernel)(P...), int64_t blocks, Split s, int threads, int smem,
                   cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.cluster), static_cast<unsigned>(blocks),
                     static_cast<unsigned>(s.segments));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
  p.fault = device_fault_word();
  if (!p.fault) return GGRN_ERR_CUDA;
  if (p.mute && k.cluster == 1) return GGRN_ERR_UNSUPPORTED;
  constexpr int kSmem = 3 * kTile * kCols * sizeof(T);
  const cudaError_t e = allow_shared_memory<forward::k_recur<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  return launch_cluster(forward::k_recur<T>, blocks, k, forward::kThreads, kSmem, s, p);
}
template <typename T>
int launch_backward(Params& p, float* sums, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width);
  const Split k = split_rows(p.q.rows, p.q.seqs, blocks, 2);
  p.segments = k.segments;
  p.fault = device_fault_word();
  if (!p.fault) return GGRN_ERR_CUDA;
  float* const da = p.da;
  if (k.segments > 1) p.da = sums;
  constexpr int kSmem = backward::stages<T>() * 4 * kTile * kCols * sizeof(T);
  const cudaError_t e = allow_shared_memory<backward::k_recur_backward<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  const int st = launch_cluster(backward::k_recur_backward<T>, blocks, k, backward::kThreads, kSmem,
                                s, p);
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
int run_kernels(Params& p, const Space& need, void* workspace, cudaStream_t s) {
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
  if (c.dtype == kF32) return run_kernels<float>(p, need, w, s);
  if (c.dtype == kF16) return run_kernels<__half>(p, need, w, s);
  return run_kernels<__nv_bfloat16>(p, need, w, s);
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
