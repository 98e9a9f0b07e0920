// ggrn_conv.cu -- the mixer's short causal convolution (depthwise, 2 to 4
// taps, bias, SiLU) over packed sequences, and its form for single tokens.
//
//   v[t, c] = bias[c] + sum_{k < W} w[c, k] * u[t - (W-1) + k, c],  out = silu(v)
//
// Bound by HBM: each input is read once and each output written once (4 bytes
// per element for 16-bit T against ~20 operations).  A thread keeps the W taps
// of one 16-byte vector of channels in registers and slides its window down a
// tile of rows, four rows of loads ahead of the ones it computes; an input is
// loaded once per thread plus W-1 rows of overlap between tiles, which come
// from L2.  The arithmetic runs on f32 pairs.  4096 x 9728 bf16: 30.0 us, 78 %
// of the rate of a plain copy (27.9 without the SiLU, whose exponential and
// reciprocal take 17 us of the special function units); f32, with an accurate
// SiLU: 53.7 us, 88 % (50.9 without it).
//
// Rows whose window reaches before their sequence (the first W-1) and the
// pool's entries belong to other CTAs of the same launch, one per sequence
// and channel block: each thread there reads its channels of the old entry,
// computes those rows and writes the new entry, so no thread reads an entry
// that another one writes.  The step form is those CTAs alone, several
// sequences to a thread (in 16-bit types the taps and the bias are ten times
// a row's bytes): 256 x 9728 bf16 6.7 us, the pool's entries being in L2.
#include <cuda_runtime.h>

#include "ggrn_mixer.cuh"

namespace ggrn {
namespace conv {

constexpr int kThreads = 64;
constexpr int kAhead = 4;  // rows of loads in flight
// CTAs of an SM: ten leave a thread 102 registers.  Prompts of 4096 x 9728
// bf16: 29.8 us with ten, 35 with nine, 44 with eleven (which spill).
constexpr int kResident = 10;
// Rows a thread slides its window over: the multiple of kAhead up to
// kMaxTileRows whose waves cost least, a tile costing its rows and
// kTileCost more (loads of the taps and the rows before the tile).  One wave
// of 52 rows against two of 24: 29.8 and 33 us in the case above.
constexpr int kMaxTileRows = 64;
constexpr int kTileCost = 6;
static_assert(kMaxTileRows <= kThreads, "a thread places one row of the tile");

struct Params {
  const void* x;
  const float* w;
  const float* bias;
  void* out;
  void* state;
  Seqs q;
  int64_t xs, os, slot_stride;
  int64_t width;      // channels
  int64_t vecs;       // channel vectors
  int64_t tiles;      // row tiles (0 in the step form)
  int tile_rows;      // a multiple of kAhead
  int step;
};

// V elements of T: a 16-byte vector, or one element where the layout does not
// allow vectors.
template <typename T, int V>
struct Vec {
  static_assert(V * sizeof(T) == 16, "a 16-byte vector");
  uint4 v;
  __device__ __forceinline__ static Vec load(const T* p) {
    return {*reinterpret_cast<const uint4*>(p)};
  }
  __device__ __forceinline__ static Vec zero() { return {make_uint4(0, 0, 0, 0)}; }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void unpack(float (&f)[V]) const { Elem<T>::unpack(v, f); }
  __device__ __forceinline__ static Vec pack(const float (&f)[V]) { return {Elem<T>::pack(f)}; }
};
template <typename T>
struct Vec<T, 1> {
  T v;
  __device__ __forceinline__ static Vec load(const T* p) { return {*p}; }
  __device__ __forceinline__ static Vec zero() {
    const float z[1] = {0.0f};
    return pack(z);
  }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = static_cast<float>(v); }
  __device__ __forceinline__ static Vec pack(const float (&f)[1]) {
    Vec r;
    Elem<T>::store1(&r.v, 0, f[0]);
    return r;
  }
};

template <typename T, int V, int W, bool SILU>
struct Taps {
  float w[W][V];
  float bias[V];
  __device__ __forceinline__ void load(const Params& p, int64_t c0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (W == 4 && V > 1) {  // vectors come with a 16-byte aligned w
        const float4 q = __ldg(reinterpret_cast<const float4*>(p.w) + c0 + i);
        w[0][i] = q.x, w[1][i] = q.y, w[2][i] = q.z, w[3][i] = q.w;
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = __ldg(p.w + (c0 + i) * W + k);
      }
      bias[i] = p.bias ? __ldg(p.bias + c0 + i) : 0.0f;
    }
  }
  // The output vector of a window (oldest first).
  __device__ __forceinline__ Vec<T, V> apply(const Vec<T, V>* win) const {
    float acc[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      win[k].unpack(u);
      if constexpr (V == 1) {
        acc[0] = fmaf(w[k][0], u[0], acc[0]);
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 2)
          fma2(acc[i], acc[i + 1], w[k][i], w[k][i + 1], u[i], u[i + 1], acc[i], acc[i + 1]);
      }
    }
    if constexpr (SILU) {
      if constexpr (V == 1) {
        acc[0] = silu<T>(acc[0]);
      } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) silu2<T>(acc[i], acc[i + 1], acc[i], acc[i + 1]);
      }
    }
    return Vec<T, V>::pack(acc);
  }
};

// The first rows of sequence i and its pool entry.
template <typename T, int V, int W, bool SILU>
__device__ __forceinline__ void head(const Params& p, const Taps<T, V, W, SILU>& taps, int64_t i,
                                     int64_t c0) {
  using Vc = Vec<T, V>;
  const T* x = static_cast<const T*>(p.x) + c0;
  T* out = static_cast<T*>(p.out) + c0;
  const int64_t slot = seq_slot(p.q, i);
  int64_t begin, end;
  seq_range(p.q, i, begin, end);
  const int64_t n = end - begin;
  T* entry = static_cast<T*>(p.state) + slot * p.slot_stride + c0;
  constexpr int M = W - 1;  // rows here
  Vc win[W - 1 + M];                   // the old entry, then the sequence's first rows
  const bool resume = slot >= 0 && seq_resumes(p.q, i);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = resume ? Vc::load(entry + j * p.width) : Vc::zero();
#pragma unroll
  for (int j = 0; j < M; ++j)
    win[W - 1 + j] = j < n ? Vc::load(x + (begin + j) * p.xs) : Vc::zero();
#pragma unroll
  for (int j = 0; j < M; ++j)
    if (j < n) taps.apply(win + j).store(out + (begin + j) * p.os);
  if (slot < 0) return;
  // the new entry: inputs n - (W-1) .. n - 1, where negative ones are the old entry's
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    Vc v;
    if (n > M) {
      v = Vc::load(x + (end - (W - 1) + j) * p.xs);
    } else {
      v = win[j];  // n == 0
#pragma unroll
      for (int m = 1; m <= M; ++m)
        if (n == m) v = win[j + m];
    }
    v.store(entry + j * p.width);
  }
}

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, kResident) k_conv(const Params p) {
  using Vc = Vec<T, V>;
  __shared__ int s_pos[kMaxTileRows];  // place of each row of the tile in its sequence; -1: of none
  pdl_wait();
  pdl_launch_dependents();
  const int64_t cv = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  const bool active = cv < p.vecs;
  const int64_t c0 = cv * V;
  Taps<T, V, W, SILU> taps;
  if (blockIdx.x >= p.tiles) {
    if (!active) return;
    taps.load(p, c0);
    head<T, V, W, SILU>(p, taps, static_cast<int64_t>(blockIdx.x) - p.tiles, c0);
    return;
  }

  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.tile_rows;
  const T* xc = static_cast<const T*>(p.x) + c0;
  T* out = static_cast<T*>(p.out) + c0;
  // win: the W-1 rows before the next ones, then those
  Vc win[W - 1 + kAhead], next[kAhead];
  if (active) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t r = r0 - (W - 1) + j;
      win[j] = r >= 0 ? Vc::load(xc + r * p.xs) : Vc::zero();
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      next[j] = r0 + j < p.q.rows ? Vc::load(xc + (r0 + j) * p.xs) : Vc::zero();
    taps.load(p, c0);
  }
  if (threadIdx.x < p.tile_rows) {
    const int64_t r = r0 + threadIdx.x;
    int pos = -1;
    if (r < p.q.rows) {
      int64_t begin = 0, end = 0;
      if (p.q.cu) {
        // the last sequence that begins at or before r
        int64_t lo = 0, hi = p.q.seqs;  // cu[lo] <= r (or lo == 0), cu[hi] > r (or hi == seqs)
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (__ldg(p.q.cu + mid) <= r) lo = mid;
          else hi = mid;
        }
        seq_range(p.q, lo, begin, end);
      } else {
        begin = r / p.q.each * p.q.each;
        end = begin + p.q.each;
      }
      if (r >= begin && r < end) pos = static_cast<int>(r - begin < W ? r - begin : W);
    }
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  if (!active) return;
#pragma unroll 1
  for (int b = 0; b < p.tile_rows; b += kAhead) {
    const int64_t rb = r0 + b;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) win[W - 1 + j] = next[j];
    if (b + kAhead < p.tile_rows) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        next[j] = rb + kAhead + j < p.q.rows ? Vc::load(xc + (rb + kAhead + j) * p.xs) : Vc::zero();
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      // a place of W-1 or more: the whole window lies in the sequence
      if (s_pos[b + j] >= W - 1) taps.apply(win + j).store(out + (rb + j) * p.os);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = win[kAhead + j];
  }
}

// The step form: SEQS sequences to a thread, all loads before the first store
// (the slots of one call are distinct).  A row without a slot is left alone.
template <typename T, int V, int W, bool SILU, int SEQS>
__global__ void __launch_bounds__(kThreads) k_conv_step(const Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t cv = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  if (cv >= p.vecs) return;
  Taps<T, V, W, SILU> taps;
  const int64_t c0 = cv * V;
  const T* x = static_cast<const T*>(p.x) + c0;
  T* out = static_cast<T*>(p.out) + c0;
  T* pool = static_cast<T*>(p.state) + c0;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * SEQS;
  Vec<T, V> win[SEQS][W];
  int64_t slot[SEQS];
#pragma unroll
  for (int k = 0; k < SEQS; ++k) slot[k] = i0 + k < p.q.seqs ? seq_slot(p.q, i0 + k) : -1;
#pragma unroll
  for (int k = 0; k < SEQS; ++k) {
    if (slot[k] < 0) continue;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      win[k][j] = Vec<T, V>::load(pool + slot[k] * p.slot_stride + j * p.width);
    win[k][W - 1] = Vec<T, V>::load(x + (i0 + k) * p.xs);
  }
  taps.load(p, c0);
#pragma unroll
  for (int k = 0; k < SEQS; ++k) {
    if (slot[k] < 0) continue;
    taps.apply(win[k]).store(out + (i0 + k) * p.os);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      win[k][j + 1].store(pool + slot[k] * p.slot_stride + j * p.width);
  }
}

// Sequences to a thread of the step form: four where that leaves two CTAs for
// each SM (256 x 9728 bf16: 6.3 us, against 9.3 with two and 17.7 with one),
// else one.
constexpr int kStepSeqs = 4;

template <typename T, int V, int W, bool SILU>
int launch_rows(Params& p, cudaStream_t s) {
  const int64_t gy = (p.vecs + kThreads - 1) / kThreads;
  int64_t gx;
  const bool many = p.step && p.q.seqs * gy >= 2 * kStepSeqs * static_cast<int64_t>(device_sms());
  if (p.step) {
    gx = many ? (p.q.seqs + kStepSeqs - 1) / kStepSeqs : p.q.seqs;
  } else {
    int best = 0;
    int64_t cost = INT64_MAX;
    const int64_t room = kResident * static_cast<int64_t>(device_sms());
    for (int t = kAhead; t <= kMaxTileRows; t += kAhead) {
      const int64_t ctas = (p.q.rows + t - 1) / t * gy;
      const int64_t c = (ctas + room - 1) / room * (t + kTileCost);
      if (c <= cost) cost = c, best = t;
    }
    p.tile_rows = best;
    p.tiles = (p.q.rows + p.tile_rows - 1) / p.tile_rows;
    gx = p.tiles + p.q.seqs;
  }
  if (gx == 0) return GGRN_OK;
  if (gx > INT32_MAX || gy > 65535) return GGRN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (!p.step) return mixer::launch(k_conv<T, V, W, SILU>, grid, kThreads, 0, s, p);
  return many ? mixer::launch(k_conv_step<T, V, W, SILU, kStepSeqs>, grid, kThreads, 0, s, p)
              : mixer::launch(k_conv_step<T, V, W, SILU, 1>, grid, kThreads, 0, s, p);
}
template <typename T, int V>
int launch_taps(Params& p, int taps, int act, cudaStream_t s) {
  const bool silu = act == GGRN_ACT_SILU;
  if (taps == 2) return silu ? launch_rows<T, V, 2, true>(p, s) : launch_rows<T, V, 2, false>(p, s);
  if (taps == 3) return silu ? launch_rows<T, V, 3, true>(p, s) : launch_rows<T, V, 3, false>(p, s);
  return silu ? launch_rows<T, V, 4, true>(p, s) : launch_rows<T, V, 4, false>(p, s);
}
template <typename T>
int launch_vec(Params& p, bool vec, int taps, int act, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  p.vecs = vec ? p.width / V : p.width;
  return vec ? launch_taps<T, V>(p, taps, act, s) : launch_taps<T, 1>(p, taps, act, s);
}

int check(const ggrn_conv_call& c, bool step, Params* p) {
  if (c.dtype != kF32 && c.dtype != kF16 && c.dtype != kBF16) return GGRN_ERR_DTYPE;
  if (c.activation != GGRN_ACT_NONE && c.activation != GGRN_ACT_SILU) return GGRN_ERR_ARG;
  if (c.width <= 0) return GGRN_ERR_SHAPE;
  if (c.taps < 2 || c.taps > 4) return GGRN_ERR_UNSUPPORTED;
  // widths whose entry does not fit in int64, or that the grid cannot hold
  if (c.width > int64_t{1} << 40) return GGRN_ERR_SHAPE;
  if (c.width > int64_t{65535} * kThreads) return GGRN_ERR_UNSUPPORTED;
  const int es = mixer::elem_bytes(c.dtype);
  const int64_t held = (c.taps - 1) * c.width;
  int st = mixer::check_seqs(c.rows, c.seqs, c.cu_seqlens, c.state, c.slots, c.resume,
                             c.state_slots, held, c.state_slot_stride, step, &p->q);
  if (st != GGRN_OK) return st;
  mixer::Buffer x, out, state, w, bias;
  if (!mixer::extent(c.x, c.rows, c.width, c.x_row_stride, es, &x) ||
      !mixer::extent(c.out, c.rows, c.width, c.out_row_stride, es, &out) ||
      !mixer::extent(c.state, c.state ? c.state_slots : 0, held, c.state_slot_stride, es, &state))
    return GGRN_ERR_SHAPE;
  if (c.rows == 0 && (!c.state || p->q.seqs == 0)) return GGRN_OK;
  if (!c.w || (c.rows > 0 && (!c.x || !c.out))) return GGRN_ERR_NULL;
  if (!mixer::aligned_to(c.x, es) || !mixer::aligned_to(c.out, es) ||
      !mixer::aligned_to(c.state, es) || !mixer::aligned_to(c.w, 4) ||
      !mixer::aligned_to(c.bias, 4))
    return GGRN_ERR_ALIGN;
  w = {c.w, c.width * c.taps * 4};
  bias = {c.bias, c.width * 4};
  const mixer::Buffer cu = {p->q.cu, (p->q.seqs + 1) * 4}, slots = {p->q.slots, p->q.seqs * 4},
                      res = {p->q.resume, p->q.seqs};
  for (const mixer::Buffer& o : {out, state})
    for (const mixer::Buffer& i : {x, w, bias, cu, slots, res})
      if (mixer::overlap(o, i)) return GGRN_ERR_OVERLAP;
  if (mixer::overlap(out, state)) return GGRN_ERR_OVERLAP;
  p->x = c.x;
  p->w = c.w;
  p->bias = c.bias;
  p->out = c.out;
  p->state = c.state;
  p->xs = c.rows > 1 ? c.x_row_stride : 0;
  p->os = c.rows > 1 ? c.out_row_stride : 0;
  p->slot_stride = c.state_slots > 1 ? c.state_slot_stride : 0;
  p->width = c.width;
  p->step = step;
  return GGRN_OK;
}

int run(const ggrn_conv_call* call, bool step, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_conv_call& c = *call;
  Params p = {};
  const int st = check(c, step, &p);
  if (st != GGRN_OK || (c.rows == 0 && (!c.state || p.q.seqs == 0))) return st;
  const int es = mixer::elem_bytes(c.dtype);
  // 16-byte vectors of channels where every row of every buffer starts on one
  const bool vec = c.width * es % 16 == 0 && mixer::aligned_to(c.x, 16) &&
                   mixer::aligned_to(c.out, 16) && mixer::aligned_to(c.state, 16) &&
                   mixer::aligned_to(c.w, 16) && p.xs * es % 16 == 0 && p.os * es % 16 == 0 &&
                   p.slot_stride * es % 16 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.dtype == kF32) return launch_vec<float>(p, vec, c.taps, c.activation, s);
  if (c.dtype == kF16) return launch_vec<__half>(p, vec, c.taps, c.activation, s);
  return launch_vec<__nv_bfloat16>(p, vec, c.taps, c.activation, s);
}

}  // namespace conv

int check_conv(const ggrn_conv_call& c, bool step) {
  conv::Params p = {};
  return conv::check(c, step, &p);
}

}  // namespace ggrn

extern "C" int ggrn_conv(const ggrn_conv_call* call, void* cuda_stream) {
  return ggrn::conv::run(call, false, cuda_stream);
}
extern "C" int ggrn_conv_step(const ggrn_conv_call* call, void* cuda_stream) {
  return ggrn::conv::run(call, true, cuda_stream);
}
