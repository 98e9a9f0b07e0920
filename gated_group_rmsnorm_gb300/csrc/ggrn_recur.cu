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
// consecutive rows of 64 channels and composes their pairs; the CTA's warps hold a
// tile of 64 rows and exchange theirs in shared memory; the CTAs of a cluster hold
// consecutive tiles and exchange theirs through distributed shared memory.  A
// cluster walks down (the gradients: up) its rows with the state in registers, so
// each input is read once and no CTA waits for another cluster.  The order of every
// sum is fixed.
//
// The backward pass needs the states again: the forward pass can keep the one
// before every 64th row (f32, 1/32 of a 16-bit tensor's bytes), from which each
// tile finds its own; without them a first launch makes them.
//
// An element takes 8 bytes of HBM forward and 14 back (16-bit T), five and eight
// operations of the special function units, and about 40 and 80 instructions.
// 4096 x 7680 bf16: 73 us forward, 177 back, against 37 and 65 for the bytes alone.
// f32: 2048 x 5120 56 us forward, 167 back (25 and 43).
// What is left is latency: an SM's schedulers issue half of the time, since a turn
// of a cluster is a chain (copies, gates, exchange, outputs) that the five (back: two)
// CTAs of the SM overlap only in part.
#include <cuda_runtime.h>

#include <atomic>
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
  __device__ __forceinline__ void get(float* f) const { f[0] = static_cast<float>(w); }
  __device__ __forceinline__ static void put(T* p, const float* f) { Elem<T>::store1(p, 0, f[0]); }
};

// ---------------------------------------------------------------------------
// Gates of a pair of elements.
//
// 16-bit T: sigmoid(z) = 1 / (1 + 2^(-z log2 e)) with the hardware's approximate
// exponential and reciprocal, both good to about 2^-22 (below 2^-126 they give 0).
// f32: see Accurate below.
//
// exp(p) - 1 = p + p^2 (..) where p > -1/4, with a polynomial through the
// Chebyshev points of that range (within 2^-26 of it), and e = 1 + that, m^2 =
// 1 - e^2 = -(e - 1)(2 + (e - 1)): neither loses digits to cancellation where
// decays are slow (an exponential that is off by an ulp to one side next to 1 is
// off by a thousand after a thousand rows), and slow channels take no second
// exponential.  FAST: no decay of the warp's channels is below exp(-1/4).
//
// The arithmetic is on pairs, and so are its constants: a loop over rows keeps them
// in registers (Constants, made by instructions that the compiler does not repeat),
// since a pair of constants costs two moves wherever it is used otherwise.
// ---------------------------------------------------------------------------
constexpr float kSeries = -0.25f;
constexpr float kC4 = 7.67176877707243e-3f, kC3 = 4.1564859449863434e-2f,
                kC2 = 1.666616052389145e-1f, kC1 = 4.999999701976776e-1f;

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Constants {
  Two c4 = held(kC4), c3 = held(kC3), c2 = held(kC2), c1 = held(kC1), one = held(1.0f),
      two = held(2.0f), minus = held(-1.0f), log2e = held(-1.4426950408889634f);
};

// exp(-z), and sigmoid(z) of that
__device__ __forceinline__ Two odds2(Two z, const Constants& k) {
  return each(mul(z, k.log2e), ex2_approx);
}
__device__ __forceinline__ Two gate_of(Two odds, const Constants& k) {
  return each(add(odds, k.one), rcp_approx);
}
__device__ __forceinline__ Two sigmoid2(Two z, const Constants& k) {
  return gate_of(odds2(z, k), k);
}
// 1 - sigmoid(z), without cancellation (where infinite odds meet a gate of 0, a 0: the
// gate is a factor of all that this is one of)
__device__ __forceinline__ Two rest_of(Two odds, Two gate) {
  float o[2], g[2];
  split(odds, o[0], o[1]), split(gate, g[0], g[1]);
  return join(__saturatef(o[0] * g[0]), __saturatef(o[1] * g[1]));
}

// From r and the channels' a: e = exp(a r), m = sqrt(1 - e^2).
template <bool FAST>
__device__ __forceinline__ void decay2(Two r, Two a, const Constants& k, Two& e, Two& m) {
  const Two p = mul(a, r);
  Two s = fma(fma(fma(fma(p, k.c4, k.c3), p, k.c2), p, k.c1), p, k.one);
  s = mul(s, p);  // e - 1
  e = add(s, k.one);
  if constexpr (!FAST) {
    float pv[2], ev[2], sv[2];
    split(p, pv[0], pv[1]), split(e, ev[0], ev[1]), split(s, sv[0], sv[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float far = ex2_approx(pv[i] * 1.4426950408889634f);
      if (!(pv[i] > kSeries)) ev[i] = far, sv[i] = far - 1.0f;
    }
    e = join(ev[0], ev[1]), s = join(sv[0], sv[1]);
  }
  m = each(mul(s, add(s, k.two)), [](float q) { return sqrt_approx(-q); });
}

// ---------------------------------------------------------------------------
// The same for f32, each result within a few roundings (u = 2^-24) of its argument's:
//   exp(-|z|)    t = -|z| log2 e rounded, m = -|z| - t ln 2 by two fma (Cody and Waite's
//                reduction, without an integer part), 2^t (1 + m): 5 u, 4 of them the
//                hardware's exponential (below 2^-126 it gives 0).
//   1 / (1 + E)  Newton's iteration once, from the hardware's reciprocal.  It is the larger
//                of sigmoid(z) and sigmoid(-z), E times it the smaller: 8 u, at both ends.
//   sqrt(q)      Newton's iteration once, from the hardware's reciprocal root.
// (CUDA's expf, division and sqrtf are as good, one element at a time and with branches:
// 2048 x 5120 took 84 us with them, 56 with these and 48 with the approximate functions
// of 16-bit T.)  Decays beyond the series take expf and expm1f.
// ---------------------------------------------------------------------------
struct Accurate {
  Two c4 = held(kC4), c3 = held(kC3), c2 = held(kC2), c1 = held(kC1), one = held(1.0f),
      two = held(2.0f), minus = held(-1.0f), half = held(0.5f), log2e = held(1.4426950408889634f),
      ln2 = held(-0.693147180559945309f), ln2_rest = held(1.904654299958e-9f);
};
template <typename T>
using ConstantsOf = typename std::conditional<Elem<T>::kExactSilu, Accurate, Constants>::type;

// sigmoid(z), and (in `rest`) 1 - sigmoid(z)
__device__ __forceinline__ Two sigmoid_accurate(Two z, const Accurate& k, Two& rest) {
  const Two a = each(z, [](float v) {  // -|z| (a NaN stays one), where E is 0 at the latest
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(-fabsf(v)), "f"(-128.0f));
    return r;
  });
  const Two t = mul(a, k.log2e);
  const Two m = fma(t, k.ln2_rest, fma(t, k.ln2, a));
  const Two e0 = each(t, ex2_approx), e = fma(e0, m, e0);
  const Two less = fma(e, k.minus, k.minus);  // -(1 + E)
  const Two r = each(less, [](float v) { return rcp_approx(-v); });
  const Two big = fma(r, fma(less, r, k.one), r), small = mul(e, big);
  float zv[2], bv[2], sv[2];
  split(z, zv[0], zv[1]), split(big, bv[0], bv[1]), split(small, sv[0], sv[1]);
  rest = join(zv[0] < 0.0f ? bv[0] : sv[0], zv[1] < 0.0f ? bv[1] : sv[1]);
  return join(zv[0] < 0.0f ? sv[0] : bv[0], zv[1] < 0.0f ? sv[1] : bv[1]);
}
__device__ __forceinline__ Two sigmoid_accurate(Two z, const Accurate& k) {
  Two rest;
  return sigmoid_accurate(z, k, rest);
}
// exp(p) and exp(p) - 1 of the halves that the series does not reach.
__device__ __noinline__ ulonglong2 decay_beyond(Two p, Two e, Two s) {
  float pv[2], ev[2], sv[2];
  split(p, pv[0], pv[1]), split(e, ev[0], ev[1]), split(s, sv[0], sv[1]);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const float v = i ? pv[1] : pv[0];
    if (v > kSeries) continue;
    const float x = expf(v), y = expm1f(v);
    if (i) ev[1] = x, sv[1] = y;
    else ev[0] = x, sv[0] = y;
  }
  return make_ulonglong2(join(ev[0], ev[1]), join(sv[0], sv[1]));
}
// e = exp(a r), m = sqrt(1 - e^2), and 1 / m (0 where m is)
__device__ __forceinline__ void decay_accurate(Two r, Two a, const Accurate& k, Two& e, Two& m,
                                               Two& over) {
  const Two p = mul(a, r);
  Two s = fma(fma(fma(fma(p, k.c4, k.c3), p, k.c2), p, k.c1), p, k.one);
  s = mul(s, p);  // e - 1
  e = add(s, k.one);
  float p0, p1;
  split(p, p0, p1);
  if (!(p0 > kSeries && p1 > kSeries)) {
    const ulonglong2 f = decay_beyond(p, e, s);
    e = f.x, s = f.y;
  }
  const Two q = mul(s, add(s, k.two));  // -m^2
  const Two y = each(q, [](float v) { return rsqrtf(-v); });
  const Two root = mul(q, y), half = mul(y, k.half);  // -m, nearly; 1 / 2m
  float qv[2], mv[2], ov[2];
  split(q, qv[0], qv[1]), split(mul(fma(fma(root, root, q), half, root), k.minus), mv[0], mv[1]);
  split(fma(fma(root, y, k.one), half, y), ov[0], ov[1]);
  m = join(qv[0] == 0.0f ? 0.0f : mv[0], qv[1] == 0.0f ? 0.0f : mv[1]);
  over = join(qv[0] == 0.0f ? 0.0f : ov[0], qv[1] == 0.0f ? 0.0f : ov[1]);
}
__device__ __forceinline__ void decay_accurate(Two r, Two a, const Accurate& k, Two& e, Two& m) {
  Two over;
  decay_accurate(r, a, k, e, m, over);
}

// ---------------------------------------------------------------------------
// Pairs (E, B): v -> E v + B, of a lane's two channels.  Where a sequence starts
// (or, for gradients, ends) among the rows of a pair, nothing comes in from before
// them: E is kCut.  (Not 0: a value that is not finite would leave its sequence.)
// CUTS: some pair may be cut.
// ---------------------------------------------------------------------------
struct Pair {
  Two e, b;
};
constexpr uint32_t kCutWord = 0xbf800000u;  // -1: decays are not negative
constexpr Two kCut = (static_cast<Two>(kCutWord) << 32) | kCutWord;
constexpr Two kOnes = 0x3f8000003f800000ull;
__device__ __forceinline__ bool is_cut(const Pair& s) {
  return static_cast<uint32_t>(s.e) == kCutWord;
}
template <bool CUTS>
__device__ __forceinline__ Two through(const Pair& s, Two v) {
  return CUTS && is_cut(s) ? s.b : fma(s.e, v, s.b);
}
// First s, then t.
template <bool CUTS>
__device__ __forceinline__ Pair compose(const Pair& s, const Pair& t) {
  if (CUTS && is_cut(t)) return t;
  return {CUTS && is_cut(s) ? kCut : mul(s.e, t.e), fma(t.e, s.b, t.b)};
}
// In shared memory: 16 bytes.
__device__ __forceinline__ Pair get_pair(const ulonglong2* p) {
  const ulonglong2 v = *p;
  return {v.x, v.y};
}
__device__ __forceinline__ void put_pair(ulonglong2* p, const Pair& s) {
  *p = make_ulonglong2(s.e, s.b);
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
__device__ __forceinline__ void put_peer(const ulonglong2* mine, uint32_t rank, Two v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(map_to_rank(smem_u32(mine), rank)), "l"(v)
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
struct alignas(16) Mail {
  ulonglong2 pair[2][kMaxCluster][32];
  int cut[2][kMaxCluster];  // (of CTAs that the cluster has not: 0)
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
  if (threadIdx.x < 2 * kMaxCluster) (&m.cut[0][0])[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&m.landed[0]), 1);
    mbar_init(smem_u32(&m.landed[1]), 1);
    m.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
}
// A whole warp sends to CTA `to`.
__device__ __forceinline__ void mail_send(Mail& m, int buf, int rank, int to, const Pair& v,
                                          bool cut) {
  const int lane = threadIdx.x & 31;
  const uint32_t bar = map_to_rank(smem_u32(&m.landed[buf]), to);
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
          map_to_rank(smem_u32(&m.pair[buf][rank][lane]), to)),
      "l"(v.e), "l"(v.b), "r"(bar)
      : "memory");
  if (lane == 0)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                     map_to_rank(smem_u32(&m.cut[buf][rank]), to)),
                 "r"(cut ? 1u : 0u), "r"(bar)
                 : "memory");
}
// One thread, before the wait: how much will land.  (Not behind a wait that ran out,
// whose phase is not over.)
__device__ __forceinline__ void mail_expect(Mail& m, int buf, int size) {
  if (!m.failed) mbar_expect_tx(smem_u32(&m.landed[buf]), static_cast<uint32_t>(size) * (32 * 16 + 4));
}
__device__ __forceinline__ void mail_wait(Mail& m, int buf, uint32_t parity) {
  const uint32_t bar = smem_u32(&m.landed[buf]);
  if (!try_phase(bar, parity)) wait_poll(bar, parity, &m.failed);
}
// The value that comes to the tiles of CTA `rank`, and (in `v`) the one behind all
// tiles of the cluster, from the one before them.
__device__ __forceinline__ Two mail_through(const Mail& m, int buf, int rank, int size, Two& v) {
  const int lane = threadIdx.x & 31;
  const int4 c0 = *reinterpret_cast<const int4*>(&m.cut[buf][0]);
  const int4 c1 = *reinterpret_cast<const int4*>(&m.cut[buf][4]);
  Two mine = v;
  if (((c0.x | c0.y) | (c0.z | c0.w)) | ((c1.x | c1.y) | (c1.z | c1.w))) {
    for (int k = 0; k < size; ++k) {
      if (k == rank) mine = v;
      v = through<true>(get_pair(&m.pair[buf][k][lane]), v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      if (k >= size) break;
      if (k == rank) mine = v;
      v = through<false>(get_pair(&m.pair[buf][k][lane]), v);
    }
  }
  return mine;
}

// ---------------------------------------------------------------------------
// Rows and their sequences.
// ---------------------------------------------------------------------------
template <int ROWS>
struct TileRows {
  uint32_t in[ROWS / 32], first[ROWS / 32], last[ROWS / 32];  // bits of the tile's rows
  int seq[ROWS];
};

// The sequence of row r: the last one that begins at or before it.
__device__ __forceinline__ int64_t seq_of_row(const Seqs& q, int64_t r, int64_t& begin,
                                              int64_t& end) {
  int64_t s = 0;
  if (q.seqs == 1) {
  } else if (q.cu) {
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

// Threads 0 .. ROWS - 1 of the CTA: row `tile` x ROWS + thread, if it is one of [lo, hi).
template <int ROWS>
__device__ __forceinline__ void place_rows(const Seqs& q, int64_t tile, int64_t lo, int64_t hi,
                                           TileRows<ROWS>* t) {
  const int64_t r = tile * ROWS + threadIdx.x;
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

// What a CTA knows of its tiles' rows: the rows of a sequence.
struct Rows {
  int64_t begin = 0, end = 0;
  // Whether tile `t` of the segment's rows [lo, hi) is whole, lies in one sequence,
  // and holds neither end of it.
  template <int ROWS>
  __device__ __forceinline__ bool inside(const Seqs& q, int64_t t, int64_t lo, int64_t hi) {
    const int64_t r0 = t * ROWS, r1 = r0 + ROWS;
    if (r0 > begin && r1 < end) return true;
    if (r0 < lo || r1 > hi) return false;
    seq_of_row(q, r0, begin, end);
    return r0 > begin && r1 < end;
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

// The state that sequence s starts from, in the lane's channels c .. (0 where it
// starts from none).
__device__ __forceinline__ Two start_state(const Params& p, int64_t s, int64_t c, int n) {
  const int64_t slot = seq_slot(p.q, s);
  if (slot < 0 || !seq_resumes(p.q, s)) return 0;
  const float* h = p.state + slot * p.slot_stride + c;
  return join(n > 0 ? h[0] : 0.0f, n > 1 ? h[1] : 0.0f);
}

// What comes to the last row of sequence s from the state behind it.
__device__ __forceinline__ Two end_gradient(const Params& p, int64_t s, int64_t c, int n) {
  if (!p.dstate) return 0;
  const float* g = p.dstate + s * p.width + c;
  return join(n > 0 ? __ldg(g) : 0.0f, n > 1 ? __ldg(g + 1) : 0.0f);
}

// Empty sequences among those of this warp (every `of`-th 32 from the `at`-th):
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
// Tiles in shared memory: rows of 64 channels of each input.
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

// The CTA's threads start to copy the ROWS rows of tile `tile` of one input into
// `to`, PITCH elements apart; rows outside [lo, hi) and channels behind the last one
// become zeros.  `whole`: there are none of either.
template <typename T, int THREADS, int ROWS, int PITCH, int BYTES>
__device__ __forceinline__ void copy_by(uint32_t to, const T* from, int64_t stride, int cols,
                                        int64_t r0, int64_t lo, int64_t hi, bool whole) {
  constexpr int ES = sizeof(T), E = BYTES / ES, ROW = kCols / E;  // chunks of a row
  constexpr int STEP = THREADS / ROW;                             // rows of a round
  static_assert(THREADS % ROW == 0 && ROWS % STEP == 0, "whole rounds");
  // (a thread's chunks lie below each other)
  const int row0 = static_cast<int>(threadIdx.x) / ROW, c = static_cast<int>(threadIdx.x) % ROW * E;
  const T* p = from + (r0 + row0) * stride + c;
  const int64_t step = STEP * stride;
  uint32_t at = to + (row0 * PITCH + c) * ES;
  if (whole) {
#pragma unroll 4
    for (int k = 0; k < ROWS / STEP; ++k, p += step, at += STEP * PITCH * ES)
      copy_async<BYTES>(at, p, BYTES);
    return;
  }
  const int left = cols - c, bytes = left <= 0 ? 0 : left < E ? left * ES : BYTES;
#pragma unroll 1
  for (int k = 0; k < ROWS / STEP; ++k, p += step, at += STEP * PITCH * ES) {
    const int64_t r = r0 + row0 + k * STEP;
    const int n = r >= lo && r < hi ? bytes : 0;
    copy_async<BYTES>(at, n ? p : from, n);
  }
}
template <typename T, int THREADS, int ROWS, int PITCH>
__device__ __forceinline__ void copy_tile(T* to, const void* base, int64_t stride, int64_t c0,
                                          int64_t width, int64_t tile, int64_t lo, int64_t hi,
                                          int chunk) {
  const T* from = static_cast<const T*>(base) + c0;
  const int64_t r0 = tile * ROWS;
  const int cols = static_cast<int>(width - c0 < kCols ? width - c0 : kCols);
  const bool whole = r0 >= lo && r0 + ROWS <= hi && cols == kCols;
  if (chunk == 16) {
    copy_by<T, THREADS, ROWS, PITCH, 16>(smem_u32(to), from, stride, cols, r0, lo, hi, whole);
  } else if (chunk == 4) {
    copy_by<T, THREADS, ROWS, PITCH, 4>(smem_u32(to), from, stride, cols, r0, lo, hi, whole);
  } else if constexpr (sizeof(T) == 2) {
    // single elements: through registers, sixteen in flight
    const int c = static_cast<int>(threadIdx.x) % kCols, row0 = static_cast<int>(threadIdx.x) / kCols;
    constexpr int STEP = THREADS / kCols, AT_ONCE = 16;
    static_assert(ROWS % (STEP * AT_ONCE) == 0, "whole rounds");
#pragma unroll 1
    for (int k = row0; k < ROWS; k += STEP * AT_ONCE) {
      T v[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int64_t r = r0 + k + i * STEP;
        Elem<T>::store1(&v[i], 0, 0.0f);
        if (r >= lo && r < hi && c < cols) v[i] = from[r * stride + c];
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) to[(k + i * STEP) * PITCH + c] = v[i];
    }
  }
}

// copy_tile of N inputs for whole tiles in 16-byte chunks, with a thread's addresses
// kept from one tile to the next.
template <typename T, int THREADS, int PITCH, int N>
struct Feed {
  static constexpr int ES = sizeof(T), E = 16 / ES, ROW = kCols / E, STEP = THREADS / ROW;
  const T* from[N];
  int64_t step[N], turn[N];  // between a thread's rows; between the CTA's tiles
  uint32_t to;
  __device__ __forceinline__ Feed(const void* const (&base)[N], const int64_t (&stride)[N],
                                  int64_t c0, T* tiles, int64_t tile, int tiles_apart) {
    const int row = static_cast<int>(threadIdx.x) / ROW, c = static_cast<int>(threadIdx.x) % ROW * E;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      from[k] = static_cast<const T*>(base[k]) + c0 + (tile * kTile + row) * stride[k] + c;
      step[k] = STEP * stride[k];
      turn[k] = tiles_apart * kTile * stride[k];
    }
    to = smem_u32(tiles + row * PITCH + c);
  }
  __device__ __forceinline__ void copy() const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const T* f = from[k];
#pragma unroll
      for (int i = 0; i < kTile / STEP; ++i, f += step[k])
        copy_async<16>(to + (k * kCols + i * STEP * PITCH) * ES, f, 16);
    }
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int k = 0; k < N; ++k) from[k] += turn[k];
  }
};

// A lane's two channels of a row in shared memory.
template <typename T>
__device__ __forceinline__ Two get2(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const Two*>(p);
  } else {
    float x, y;
    Elem<T>::unpack2(*reinterpret_cast<const uint32_t*>(p), x, y);
    return join(x, y);
  }
}
// An address that goes down (or up) rows.  The step is kept in bytes: the compiler
// would scale the elements' number again at every row.
template <typename T>
struct Down {
  char* at;
  int64_t step;
  __device__ __forceinline__ Down(void* base, int64_t row, int64_t stride, int64_t c, int way) {
    step = stride * static_cast<int64_t>(sizeof(T));
    at = static_cast<char*>(base) + row * step + c * static_cast<int64_t>(sizeof(T));
    step *= way;
    asm volatile("" : "+l"(step));
  }
  __device__ __forceinline__ T* operator*() const { return reinterpret_cast<T*>(at); }
  __device__ __forceinline__ void next() { at += step; }
};
// Stores both channels, or the first `cols` of them.
template <typename T>
__device__ __forceinline__ void put2(T* p, Two v) {
  float f[2];
  split(v, f[0], f[1]);
  Raw<T, 2>::put(p, f);
}
template <typename T>
__device__ __forceinline__ void put_some(T* p, Two v, int cols) {
  float x, y;
  split(v, x, y);
  if (cols > 0) Elem<T>::store1(p, 0, x);
  if (cols > 1) Elem<T>::store1(p, 1, y);
}

// What a CTA knows for all of its tiles.
struct Place {
  int64_t lo, hi;   // rows of its segment
  int64_t c0, c;    // first channel of the CTA and of the lane
  int cols;         // the lane's channels (0 to 2)
  int rank, size;   // in its cluster
  Two a;
  bool fast;        // see decay2
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
  const float a0 = w.cols > 0 ? __ldg(p.a + w.c) : 0.0f, a1 = w.cols > 1 ? __ldg(p.a + w.c + 1) : 0.0f;
  w.a = join(a0, a1);
  w.fast = __all_sync(0xffffffffu, a0 > kSeries && a1 > kSeries);
  return w;
}
// ---------------------------------------------------------------------------
// Prompts.  Four warps of sixteen rows each, five CTAs to an SM (f32: four).  A row of
// the tile in shared memory holds x, the input gate and the decay gate of 64
// channels; e and b take their place (512 bytes a row, which f32's inputs need
// anyway), so that the loops over rows stay rolled: unrolled, with e and b in
// registers, they were larger than the instruction cache, which a third of all
// stalls waited for.  One CTA of twelve warps to an SM, its next tile's copies under
// way meanwhile, took 100 us for 4096 x 7680 in bf16 where this takes 73: a CTA's
// stages wait for each other, and other CTAs fill the gaps better.
// ---------------------------------------------------------------------------
namespace forward {

constexpr int R = 16;
constexpr int kAtOnce = 4;  // rows of a loop's turn
constexpr int W = 4, kThreads = 32 * W;
static_assert(R * W == kTile, "a tile's rows");
template <typename T>
constexpr int pitch() {  // elements between rows of the tile
  return (sizeof(T) == 2 ? 4 : 3) * kCols;
}
template <typename T>
constexpr int smem() {
  return kTile * pitch<T>() * static_cast<int>(sizeof(T));
}

struct Shared {
  ulonglong2 pair[W][32];
  Mail mail;
  TileRows<kTile> rows;
};

template <typename T>
__device__ __noinline__ void fetch(const Params& p, int64_t lo, int64_t hi, int64_t c0, T* to,
                                   int64_t tile) {
#pragma unroll 1
  for (int k = 0; k < 3; ++k)
    copy_tile<T, kThreads, kTile, pitch<T>()>(to + k * kCols, k == 0 ? p.x : k == 1 ? p.ig : p.rg,
                                              k == 0 ? p.xs : k == 1 ? p.is : p.rs, c0, p.width,
                                              tile, lo, hi, p.chunk);
}

// One tile.  INSIDE: all of its rows are those of one sequence, neither its first
// nor its last.  FAST: see decay2 (f32: true).  Takes the state before the cluster's
// tiles and gives the one behind them.
template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ Two turn_of(const Params& p, const Place& w, Shared& sh, T* tiles,
                                       int64_t tile, int64_t turn, Two state,
                                       const ConstantsOf<T>& con) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int buf = turn & 1;
  const uint32_t parity = turn >> 1 & 1;
  constexpr bool kAccurate = Elem<T>::kExactSilu;
  T* const mine = tiles + warp * R * pitch<T>();
  const auto& t = sh.rows;
  const auto bits = [&](const uint32_t* of) {
    return INSIDE ? 0u : of[warp >> 1] >> (warp & 1) * 16 & 0xffffu;
  };
  const uint32_t in = bits(t.in), first = bits(t.first), last = bits(t.last);
  const auto pair_of = [&](int j) {
    return reinterpret_cast<ulonglong2*>(mine + j * pitch<T>()) + lane;
  };
  // e and b of the warp's rows, and the pair of all of them
  // (off the loop that nearly all tiles take, short code counts for more)
  constexpr int kAtOnce = INSIDE && FAST ? forward::kAtOnce : 2;
  Pair all = {kOnes, 0};
#pragma unroll 1
  for (int j0 = 0; j0 < R; j0 += kAtOnce) {
    Two x[kAtOnce], gi[kAtOnce], gr[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const T* row = mine + (j0 + k) * pitch<T>() + lane * 2;
      x[k] = get2(row), gi[k] = get2(row + kCols), gr[k] = get2(row + 2 * kCols);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      Pair s;
      Two m;
      if constexpr (kAccurate) {
        decay_accurate(sigmoid_accurate(gr[k], con), w.a, con, s.e, m);
        s.b = mul(mul(m, sigmoid_accurate(gi[k], con)), x[k]);
      } else {
        decay2<FAST>(sigmoid2(gr[k], con), w.a, con, s.e, m);
        s.b = mul(mul(m, sigmoid2(gi[k], con)), x[k]);
      }
      if constexpr (!INSIDE) {
        if (!(in >> (j0 + k) & 1)) s = {kOnes, 0};
        if (first >> (j0 + k) & 1)
          s = {kCut, fma(s.e, start_state(p, t.seq[warp * R + j0 + k], w.c, w.cols), s.b)};
      }
      all = compose<!INSIDE>(all, s);
      put_pair(pair_of(j0 + k), s);
    }
  }
  put_pair(&sh.pair[warp][lane], all);
  __syncthreads();

  // the state before this warp's rows
  Two h = state;
  if (w.size == 1) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (k == warp) h = state;
      state = through<!INSIDE>(get_pair(&sh.pair[k][lane]), state);
    }
  } else {
    Pair whole = get_pair(&sh.pair[0][lane]);
#pragma unroll
    for (int k = 1; k < W; ++k) whole = compose<!INSIDE>(whole, get_pair(&sh.pair[k][lane]));
    if (threadIdx.x == 0) mail_expect(sh.mail, buf, w.size);
    const bool cut = !INSIDE && (t.first[0] | t.first[1]) != 0;
    if (!p.mute)
      for (int k = warp; k < w.size; k += W) mail_send(sh.mail, buf, w.rank, k, whole, cut);
    mail_wait(sh.mail, buf, parity);
    h = mail_through(sh.mail, buf, w.rank, w.size, state);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      if (k < warp) h = through<!INSIDE>(get_pair(&sh.pair[k][lane]), h);
  }
  const int64_t row0 = tile * kTile + warp * R;
  if (p.saved && warp == 0 && row0 >= w.lo && row0 < w.hi)
    put_some(p.saved + tile * p.width + w.c, h, w.cols);
  Down<T> at(p.out, row0, p.os, w.c, 1);
  const bool pairs = p.pairs && w.c0 + kCols <= p.width;
  if (INSIDE && !p.out) {
    // (only the states to be kept are wanted)
  } else if (INSIDE && pairs) {
    // (the loop that nearly all tiles of a call take)
#pragma unroll 1
    for (int j0 = 0; j0 < R; j0 += kAtOnce) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k, at.next()) {
        h = through<false>(get_pair(pair_of(j0 + k)), h);
        put2(*at, h);
      }
    }
  } else {
#pragma unroll 1
    for (int j = 0; j < R; ++j, at.next()) {
      h = through<!INSIDE>(get_pair(pair_of(j)), h);
      if (p.out && (INSIDE || (in >> j & 1))) {
        if (pairs) put2(*at, h);
        else put_some(*at, h, w.cols);
      }
      if (!INSIDE && p.keep_state && (last >> j & 1)) {
        const int64_t slot = seq_slot(p.q, t.seq[warp * R + j]);
        if (slot >= 0) put_some(p.state + slot * p.slot_stride + w.c, h, w.cols);
      }
    }
  }
  __syncthreads();  // (the next tile's copies and search write what was read here)
  return state;
}
// The forms that few tiles take, out of the way of the loop's instructions and
// registers.
template <typename T, bool INSIDE, bool FAST>
__device__ __noinline__ Two turn_apart(const Params& p, Place w, Shared& sh, T* tiles,
                                       int64_t tile, int64_t turn, Two state) {
  return turn_of<T, INSIDE, FAST>(p, w, sh, tiles, tile, turn, state, ConstantsOf<T>());
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4)
    k_recur(const __grid_constant__ Params p) {
  extern __shared__ uint4 s_tile[];
  __shared__ Shared sh;
  T* const tiles = reinterpret_cast<T*>(s_tile);
  pdl_wait();
  pdl_launch_dependents();
  mail_init(sh.mail);
  all_arrive();  // (every CTA has begun before another one writes to it)
  const Place w = find_place(p);
  const int64_t tile0 = w.lo / kTile, count = w.hi > w.lo ? (w.hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (count + w.size - 1) / w.size;
  int64_t tile = tile0 + w.rank;
  Feed<T, kThreads, pitch<T>(), 3> feed({p.x, p.ig, p.rg}, {p.xs, p.is, p.rs}, w.c0, tiles, tile,
                                        w.size);
  const bool wide = p.chunk == 16 && w.c0 + kCols <= p.width;
  all_wait();

  const ConstantsOf<T> con;
  Two state = 0;  // before the cluster's tiles
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn, tile += w.size) {
    if (wide && tile * kTile >= w.lo && (tile + 1) * kTile <= w.hi) feed.copy();
    else fetch(p, w.lo, w.hi, w.c0, tiles, tile);
    feed.advance();
    const bool inside = known.inside<kTile>(p.q, tile, w.lo, w.hi);
    if (!inside && threadIdx.x < kTile) place_rows<kTile>(p.q, tile, w.lo, w.hi, &sh.rows);
    copies_wait();
    __syncthreads();
    if constexpr (Elem<T>::kExactSilu) {
      if (inside) state = turn_of<T, true, true>(p, w, sh, tiles, tile, turn, state, con);
      else state = turn_apart<T, false, true>(p, w, sh, tiles, tile, turn, state);
    } else {
      if (inside && w.fast) state = turn_of<T, true, true>(p, w, sh, tiles, tile, turn, state, con);
      else if (inside) state = turn_apart<T, true, false>(p, w, sh, tiles, tile, turn, state);
      else if (w.fast) state = turn_apart<T, false, true>(p, w, sh, tiles, tile, turn, state);
      else state = turn_apart<T, false, false>(p, w, sh, tiles, tile, turn, state);
    }
  }
  if (p.keep_state) {
    each_empty(p.q, (static_cast<int64_t>(blockIdx.z) * w.size + w.rank) * W + (threadIdx.x >> 5),
               static_cast<int64_t>(w.size) * p.segments * W, [&](int64_t s) {
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
// Gradients.  Eight warps of eight rows each; the cluster's tiles go from the last
// rows to the first, rank 0 has the last of them.  What a row needs again on the way
// back (e, m, both gates, the state before it) lies in shared memory behind its
// inputs, so that the first loop over rows stays rolled, as in the forward pass.  (With
// these in registers and all loops unrolled 4096 x 7680 in bf16 took 171 us, against 175
// then, and 1025 x 1001 in f32 61, against 30.  Of what lies in shared memory, the loops
// behind the exchange gain by it: 177 us, 181 by four rows.)
// ---------------------------------------------------------------------------
namespace backward {

constexpr int W = 8, R = kTile / W, kThreads = 32 * W;
constexpr int kAtOnce = 4;  // rows of a loop's turn
static_assert(W >= kMaxCluster, "a warp to each CTA that the tile's pair goes to");

// A row of the tile, in bytes: x, dout, the input gate, the decay gate; then, of each lane,
//   16-bit T  (e, m); the gates' odds exp(-z), from which i, r, 1 - i and 1 - r come again
//             (1 - i of the rounded i has no digit left at logits of 16); b, later the
//             state before the row, in the place of the gates' logits
//   f32       (e, m i), in the place of the gates' logits; (r, 1 - r);
//             (m i x (1 - i), -i x e r / m); b, later the state, in the place of x
template <typename T>
struct Row {
  static constexpr int ES = sizeof(T), kRaw = 4 * kCols * ES, kLogits = 2 * kCols * ES;
  static constexpr int kDecay = ES == 4 ? kLogits : kRaw, kGates = ES == 4 ? kRaw : kRaw + 512,
                       kTerms = kRaw + 512, kState = ES == 4 ? 0 : kLogits;
  static constexpr int kPitch = kRaw + 1024;
};
template <typename T>
constexpr int smem() {
  return kTile * Row<T>::kPitch;
}

struct Shared {
  ulonglong2 down[W][32];  // pairs of states
  ulonglong2 up[W][32];    // pairs of gradients
  Mail mail;
  TileRows<kTile> rows;
};

template <typename T>
__device__ __noinline__ void fetch(const Params& p, int64_t lo, int64_t hi, int64_t c0, T* to,
                                   int64_t tile) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k)
    copy_tile<T, kThreads, kTile, Row<T>::kPitch / static_cast<int>(sizeof(T))>(
        to + k * kCols, k == 0 ? p.x : k == 1 ? p.dout : k == 2 ? p.ig : p.rg,
        k == 0 ? p.xs : k == 1 ? p.gs : k == 2 ? p.is : p.rs, c0, p.width, tile, lo, hi, p.chunk);
}

struct Carry {
  Two g;   // the gradient of the state behind the cluster's tiles
  Two da;
};

template <typename T, bool INSIDE, bool FAST>
__device__ __forceinline__ Carry turn_of(const Params& p, const Place& w, Shared& sh, T* tiles,
                                         int64_t tile, int64_t turn, Carry carry,
                                         const ConstantsOf<T>& con) {
  using L = Row<T>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int buf = turn & 1;
  const uint32_t parity = turn >> 1 & 1;
  char* const mine = reinterpret_cast<char*>(tiles) + warp * R * L::kPitch;
  const TileRows<kTile>& t = sh.rows;
  const auto raw = [&](int j, int k) {
    return get2(reinterpret_cast<const T*>(mine + j * L::kPitch) + k * kCols + lane * 2);
  };
  const auto decay_at = [&](int j) {
    return reinterpret_cast<ulonglong2*>(mine + j * L::kPitch + L::kDecay) + lane;
  };
  const auto gates_at = [&](int j) {
    return reinterpret_cast<ulonglong2*>(mine + j * L::kPitch + L::kGates) + lane;
  };
  const auto terms_at = [&](int j) {
    return reinterpret_cast<ulonglong2*>(mine + j * L::kPitch + L::kTerms) + lane;
  };
  const auto state_at = [&](int j) {
    return reinterpret_cast<Two*>(mine + j * L::kPitch + L::kState) + lane;
  };
  Two h = 0;  // the state before the tile, as it was kept
  if (tile * kTile >= w.lo) {
    const float* kept = p.saved + tile * p.width + w.c;
    h = join(w.cols > 0 ? __ldg(kept) : 0.0f, w.cols > 1 ? __ldg(kept + 1) : 0.0f);
  }
  const auto bits = [&](const uint32_t* of) {
    return INSIDE ? 0u : of[warp >> 2] >> (warp & 3) * R & 0xffu;
  };
  const uint32_t in = bits(t.in), first = bits(t.first), last = bits(t.last);

  constexpr int kAtOnce = INSIDE && FAST ? backward::kAtOnce : 2;
  Pair down = {kOnes, 0};
  Two through_e = kOnes, up = 0;  // the rows' gradients as they come out before the first one
  bool ended = false;             // (behind a last row nothing comes through)
  constexpr bool kAccurate = Elem<T>::kExactSilu;
#pragma unroll 1
  for (int j0 = 0; j0 < R; j0 += kAtOnce) {
    Two x[kAtOnce], g[kAtOnce], zi[kAtOnce], zr[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      x[k] = raw(j0 + k, 0), g[k] = raw(j0 + k, 1), zi[k] = raw(j0 + k, 2), zr[k] = raw(j0 + k, 3);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int j = j0 + k;
      Two e, m, b;
      if constexpr (kAccurate) {
        Two ci, cr, over;
        const Two si = sigmoid_accurate(zi[k], con, ci), sr = sigmoid_accurate(zr[k], con, cr);
        decay_accurate(sr, w.a, con, e, m, over);
        const Two mi = mul(m, si);
        b = mul(mi, x[k]);
        *decay_at(j) = make_ulonglong2(e, mi);
        *gates_at(j) = make_ulonglong2(sr, cr);
        *terms_at(j) = make_ulonglong2(
            mul(b, ci), mul(mul(mul(si, x[k]), e), mul(mul(over, sr), con.minus)));
      } else {
        const Two oi = odds2(zi[k], con), od = odds2(zr[k], con);
        decay2<FAST>(gate_of(od, con), w.a, con, e, m);
        b = mul(mul(m, gate_of(oi, con)), x[k]);
        *decay_at(j) = make_ulonglong2(e, m);
        *gates_at(j) = make_ulonglong2(oi, od);
      }
      *state_at(j) = b;
      // (what is kept of a row of no sequence is not used)
      if (!INSIDE && !(in >> j & 1)) e = kOnes, b = 0, g[k] = 0;
      if (!INSIDE && (last >> j & 1))
        g[k] = add(g[k], end_gradient(p, t.seq[warp * R + j], w.c, w.cols));
      if (!INSIDE && (first >> j & 1))
        down = {kCut, fma(e, start_state(p, t.seq[warp * R + j], w.c, w.cols), b)};
      else
        down = compose<!INSIDE>(down, {e, b});
      if (INSIDE || !ended) {
        through_e = mul(through_e, e);
        up = fma(through_e, g[k], up);
      }
      if (!INSIDE && (last >> j & 1)) ended = true;
    }
  }
  put_pair(&sh.down[warp][lane], down);
  put_pair(&sh.up[warp][lane], {ended ? kCut : through_e, up});
  __syncthreads();
  // the pair of the rows behind this warp's in the tile, and of the whole tile
  Pair behind = {kOnes, 0}, whole = get_pair(&sh.up[W - 1][lane]);
#pragma unroll
  for (int k = W - 2; k >= 0; --k) {
    if (k == warp) behind = whole;
    whole = compose<!INSIDE>(whole, get_pair(&sh.up[k][lane]));
  }
  if (w.size > 1) {
    if (threadIdx.x == 0) mail_expect(sh.mail, buf, w.size);
    const bool cut = !INSIDE && (t.last[0] | t.last[1]) != 0;
    if (warp < w.size) mail_send(sh.mail, buf, w.rank, warp, whole, cut);
  }
  // the states before each row, meanwhile
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    if (k < warp) h = through<!INSIDE>(get_pair(&sh.down[k][lane]), h);
#pragma unroll (INSIDE ? 8 : 1)
  for (int j = 0; j < R; ++j) {
    if (!INSIDE && (first >> j & 1)) h = start_state(p, t.seq[warp * R + j], w.c, w.cols);
    const Two b = *state_at(j), e = decay_at(j)->x;
    *state_at(j) = h;
    if (INSIDE || (in >> j & 1)) h = fma(e, h, b);
  }
  // the gradient that comes to this warp's last row from the rows behind it
  Two gc = carry.g;
  if (w.size > 1) {
    mail_wait(sh.mail, buf, parity);
    gc = mail_through(sh.mail, buf, w.rank, w.size, carry.g);
  } else {
    carry.g = through<!INSIDE>(whole, carry.g);
  }
  gc = through<!INSIDE>(behind, gc);

  const int64_t row0 = tile * kTile + warp * R;
  Down<T> dx_at(p.dx, row0 + R - 1, p.dxs, w.c, -1), di_at(p.dig, row0 + R - 1, p.dis, w.c, -1),
      dr_at(p.drg, row0 + R - 1, p.drs, w.c, -1);
  const bool pairs = p.pairs && w.c0 + kCols <= p.width;
  constexpr int kLast = INSIDE ? 8 : 2;
#pragma unroll 1
  for (int j0 = R - kLast; j0 >= 0; j0 -= kLast) {
#pragma unroll
    for (int k = kLast - 1; k >= 0; --k) {
      const int j = j0 + k;
      Two g = raw(j, 1);
      if (!INSIDE && (last >> j & 1))
        g = add(g, end_gradient(p, t.seq[warp * R + j], w.c, w.cols));
      else
        g = add(g, gc);
      // dx = g m i,  di = dx x (1 - i),  d = g e (h r - i x e r / m),  dr = d a (1 - r)
      const ulonglong2 em = *decay_at(j), gates = *gates_at(j);
      const Two eg = mul(em.x, g);
      Two dx, di, d, rest;
      if constexpr (kAccurate) {
        const ulonglong2 terms = *terms_at(j);
        rest = gates.y;
        dx = mul(em.y, g), di = mul(terms.x, g);
        d = mul(fma(*state_at(j), gates.x, terms.y), eg);
      } else {
        const Two e = em.x, m = em.y, x = raw(j, 0);
        const Two si = gate_of(gates.x, con), sr = gate_of(gates.y, con);
        rest = rest_of(gates.y, sr);
        dx = mul(mul(m, si), g), di = mul(mul(dx, x), rest_of(gates.x, si));
        const Two over = each(m, [](float v) {
          return v > 0.0f ? -rcp_approx(v) : 0.0f;
        });
        d = mul(fma(mul(mul(si, x), e), mul(over, sr), mul(*state_at(j), sr)), eg);
      }
      Two dr = mul(mul(d, w.a), rest);
      if (INSIDE || (in >> j & 1)) {
        carry.da = add(carry.da, d);
        gc = eg;
      } else {  // a row of no sequence
        dx = di = dr = 0;
      }
      if (INSIDE || (row0 + j >= w.lo && row0 + j < w.hi)) {
        if (pairs) {
          put2(*dx_at, dx), put2(*di_at, di), put2(*dr_at, dr);
        } else {
          put_some(*dx_at, dx, w.cols), put_some(*di_at, di, w.cols), put_some(*dr_at, dr, w.cols);
        }
      }
      dx_at.next(), di_at.next(), dr_at.next();
      if (!INSIDE && p.dinitial && (first >> j & 1)) {
        const int64_t s = t.seq[warp * R + j];
        const bool resumes = seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
        put_some(p.dinitial + s * p.width + w.c, resumes ? gc : 0, w.cols);
      }
    }
  }
  __syncthreads();  // (the next tile's copies and search write what was read here)
  return carry;
}
template <typename T, bool INSIDE, bool FAST>
__device__ __noinline__ Carry turn_apart(const Params& p, Place w, Shared& sh, T* tiles,
                                         int64_t tile, int64_t turn, Carry carry) {
  return turn_of<T, INSIDE, FAST>(p, w, sh, tiles, tile, turn, carry, ConstantsOf<T>());
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    k_recur_backward(const __grid_constant__ Params p) {
  extern __shared__ uint4 s_tile[];
  __shared__ Shared sh;
  T* const tiles = reinterpret_cast<T*>(s_tile);
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  mail_init(sh.mail);
  all_arrive();  // (every CTA has begun before another one writes to it)
  const Place w = find_place(p);
  const int64_t tile0 = w.lo / kTile, count = w.hi > w.lo ? (w.hi + kTile - 1) / kTile - tile0 : 0;
  const int64_t turns = (count + w.size - 1) / w.size;
  int64_t tile = tile0 + count - 1 - w.rank;
  Feed<T, kThreads, Row<T>::kPitch / static_cast<int>(sizeof(T)), 4> feed(
      {p.x, p.dout, p.ig, p.rg}, {p.xs, p.gs, p.is, p.rs}, w.c0, tiles, tile, -w.size);
  const bool wide = p.chunk == 16 && w.c0 + kCols <= p.width;
  all_wait();

  const ConstantsOf<T> con;
  Carry carry = {0, 0};
  Rows known;
  for (int64_t turn = 0; turn < turns; ++turn, tile -= w.size) {
    if (wide && tile * kTile >= w.lo && (tile + 1) * kTile <= w.hi) feed.copy();
    else fetch(p, w.lo, w.hi, w.c0, tiles, tile);
    feed.advance();
    const bool inside = known.inside<kTile>(p.q, tile, w.lo, w.hi);
    if (!inside && threadIdx.x < kTile) place_rows<kTile>(p.q, tile, w.lo, w.hi, &sh.rows);
    copies_wait();
    __syncthreads();
    if constexpr (Elem<T>::kExactSilu) {
      if (inside) carry = turn_of<T, true, true>(p, w, sh, tiles, tile, turn, carry, con);
      else carry = turn_apart<T, false, true>(p, w, sh, tiles, tile, turn, carry);
    } else {
      if (inside && w.fast) carry = turn_of<T, true, true>(p, w, sh, tiles, tile, turn, carry, con);
      else if (inside) carry = turn_apart<T, true, false>(p, w, sh, tiles, tile, turn, carry);
      else if (w.fast) carry = turn_apart<T, false, true>(p, w, sh, tiles, tile, turn, carry);
      else carry = turn_apart<T, false, false>(p, w, sh, tiles, tile, turn, carry);
    }
  }
  if (p.dinitial) {
    each_empty(p.q, (static_cast<int64_t>(blockIdx.z) * w.size + w.rank) * W + warp,
               static_cast<int64_t>(w.size) * p.segments * W, [&](int64_t s) {
                 const bool keep = p.dstate && seq_slot(p.q, s) >= 0 && seq_resumes(p.q, s);
                 for (int v = 0; v < w.cols; ++v) {
                   const int64_t k = s * p.width + w.c + v;
                   p.dinitial[k] = keep ? __ldg(p.dstate + k) : 0.0f;
                 }
               });
  }
  // da: the warps' sums, then the CTAs' in rank 0
  __syncthreads();
  sh.up[warp][lane].x = carry.da;
  __syncthreads();
  if (warp == 0) {
    Two t = sh.up[0][lane].x;
    for (int k = 1; k < W; ++k) t = add(t, sh.up[k][lane].x);
    put_peer(&sh.mail.pair[turns & 1][w.rank][lane], 0, t);
    if (lane == 0 && sh.mail.failed) atomicOr(p.fault, kFaultRecurWait);
  }
  all_arrive();
  all_wait();
  if (w.rank == 0 && warp == 0) {
    Two t = 0;
    for (int k = 0; k < w.size; ++k) t = add(t, sh.mail.pair[turns & 1][k][lane].x);
    put_some(p.da + blockIdx.z * p.width + w.c, t, w.cols);
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
  float* state = p.state + slot * p.slot_stride + c;
  Raw<T, V> xr, ir, rr;
  xr.load(static_cast<const T*>(p.x) + row * p.xs + c);
  ir.load(static_cast<const T*>(p.ig) + row * p.is + c);
  rr.load(static_cast<const T*>(p.rg) + row * p.rs + c);
  float x[2] = {0.0f, 0.0f}, gi[2] = {0.0f, 0.0f}, gr[2] = {0.0f, 0.0f}, a[2] = {0.0f, 0.0f},
        h[2] = {0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    a[v] = __ldg(p.a + c + v);
    h[v] = state[v];
  }
  xr.get(x), ir.get(gi), rr.get(gr);
  const Two zi = join(gi[0], gi[1]), zr = join(gr[0], gr[1]), av = join(a[0], a[1]);
  const ConstantsOf<T> con;
  Two e, m, si;
  if constexpr (Elem<T>::kExactSilu) {
    si = sigmoid_accurate(zi, con);
    decay_accurate(sigmoid_accurate(zr, con), av, con, e, m);
  } else {
    si = sigmoid2(zi, con);
    decay2<false>(sigmoid2(zr, con), av, con, e, m);
  }
  split(fma(e, join(h[0], h[1]), mul(mul(m, si), join(x[0], x[1]))), h[0], h[1]);
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = h[v];
  Raw<T, V>::put(static_cast<T*>(p.out) + row * p.os + c, h);
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
// How the tiles of a call are shared out: CTAs of a cluster, and segments.
struct Split {
  int cluster = 1, segments = 1;
};

// Clusters of k CTAs that run at the same time, a kernel's CTAs `resident` to an SM:
// as the device says (a cluster lies within a group of SMs, which leaves places
// over), once for each kernel, k and device; without a device its places' number.
template <auto kernel>
int64_t clusters_at_once(int threads, int smem, int resident, int k) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return device_sms() * static_cast<int64_t>(resident) / k;
  }
  int n = known[dev][k].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(k), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(k);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = device_sms() * resident / k;
    }
    known[dev][k].store(n, std::memory_order_relaxed);
  }
  return n;
}

// The largest cluster of which those of all blocks of channels run at the same
// time: one more CTA in each makes a second round of clusters (4096 x 7680 bf16: 92
// us with four CTAs, 80 with five, 74 with six, of which 120 fit, and 105 with
// seven).  Where eight leave room, packed sequences are cut into segments.
template <auto kernel>
Split split_rows(int threads, int smem, int resident, int64_t rows, int64_t seqs,
                 int64_t blocks) {
  Split s;
  const int64_t tiles = (rows + kTile - 1) / kTile;
  const int64_t most = tiles < kMaxCluster ? (tiles < 1 ? 1 : tiles) : kMaxCluster;
  int64_t room = clusters_at_once<kernel>(threads, smem, resident, 1);
  for (int k = 2; k <= most; ++k) {
    const int64_t n = clusters_at_once<kernel>(threads, smem, resident, k);
    if (blocks <= n) s.cluster = k, room = n;
  }
  const int64_t want = room / blocks;
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
  constexpr int kSmem = forward::smem<T>();
  const cudaError_t e = allow_shared_memory<forward::k_recur<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  const Split k = split_rows<forward::k_recur<T>>(forward::kThreads, kSmem, sizeof(T) == 2 ? 5 : 4,
                                                  p.q.rows, p.q.seqs, blocks);
  p.segments = k.segments;
  p.fault = device_fault_word();
  if (!p.fault) return GGRN_ERR_CUDA;
  if (p.mute && k.cluster == 1) return GGRN_ERR_UNSUPPORTED;
  return launch_cluster(forward::k_recur<T>, blocks, k, forward::kThreads, kSmem, s, p);
}
template <typename T>
Split split_backward(int64_t rows, int64_t seqs, int64_t width) {
  constexpr int kSmem = backward::smem<T>();
  if (allow_shared_memory<backward::k_recur_backward<T>>(kSmem) != cudaSuccess) cudaGetLastError();
  return split_rows<backward::k_recur_backward<T>>(
      backward::kThreads, kSmem, sizeof(T) == 2 ? 2 : 1, rows, seqs, blocks_of(width));
}
template <typename T>
int launch_backward(Params& p, float* sums, cudaStream_t s) {
  const int64_t blocks = blocks_of(p.width);
  constexpr int kSmem = backward::smem<T>();
  const cudaError_t e = allow_shared_memory<backward::k_recur_backward<T>>(kSmem);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  const Split k = split_backward<T>(p.q.rows, p.q.seqs, p.width);
  p.segments = k.segments;
  p.fault = device_fault_word();
  if (!p.fault) return GGRN_ERR_CUDA;
  float* const da = p.da;
  if (k.segments > 1) p.da = sums;
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

// The most columns of a call, as ggrn.h gives it: half of what the blocks of 64 channels on
// a grid's second axis could hold (the step form's have 128 at least).
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
  const auto matrix = [&](const mixer::Buffer& b, int64_t stride) {
    return mixer::columns(b, c.rows, c.width, stride, es);
  };
  const auto vector = [](const void* q, int64_t n) { return mixer::Columns{{q, n}, 0, 0}; };
  const int64_t kept = (c.rows + kTile - 1) / kTile * c.width * 4;
  if (mixer::outputs_overlap(
          {matrix(out, c.out_row_stride), mixer::Columns{state, 0, 0}, vector(saved_p, kept)},
          {matrix(x, c.x_row_stride), matrix(ig, c.input_gate_row_stride),
           matrix(rg, c.decay_gate_row_stride), vector(c.a, c.width * 4),
           vector(p->q.cu, (p->q.seqs + 1) * 4), vector(p->q.slots, p->q.seqs * 4),
           vector(p->q.resume, p->q.seqs)}))
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

int run(const ggrn_recur_call* call, bool step, void* stream, bool mute = false) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_recur_call& c = *call;
  Params p = {};
  const int st = check(c, step, &p);
  if (mute) {
    if (st != GGRN_OK) return st;
    if (c.state || c.rows == 0) return GGRN_ERR_UNSUPPORTED;
    p.mute = 1;
    p.out = nullptr;
    p.saved = nullptr;
  }
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
  const Split k = c.dtype == kF32   ? split_backward<float>(c.rows, c.seqs, c.width)
                  : c.dtype == kF16 ? split_backward<__half>(c.rows, c.seqs, c.width)
                                    : split_backward<__nv_bfloat16>(c.rows, c.seqs, c.width);
  const int64_t most = k.segments;
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
extern "C" int ggrn_selftest_recur_timeout(const ggrn_recur_call* call, void* cuda_stream) {
  return ggrn::recur::run(call, false, cuda_stream, /*mute=*/true);
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
