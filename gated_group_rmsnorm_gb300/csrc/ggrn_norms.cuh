// ggrn_norms.cuh -- layer norm and the backward passes of layer norm and of the
// gated group-RMSNorm.
//
// All four are reductions over a group of columns of a row (layer norm: the
// whole row) and an elementwise pass over the same group, bound by HBM: a group
// is loaded once and stays in registers between the two.  The gradient of the
// weight sums over rows instead, so a thread keeps the columns it owns while
// its CTA goes down the rows, and carries their sums in registers; what is left
// is one partial sum for each CTA and column, which k_column_sum adds up in
// order.
//
// With d = x - mean, q = mean(d^2), n = rsqrt(q + eps), u = dout w:
//   layer norm           out = d n w + b
//   its gradients        dx = n (u - mean(u) - d n^2 mean(u d)),  dw += dout d n,  db += dout
// and with v = y silu(z), n = rsqrt(mean(v^2) + eps), s' the slope of silu:
//   gated norm, MAMBA2   dv = n (u - v n^2 mean(u v)),  dy = dv silu(z),  dz = dv y s',
//                        dw += dout v n
//   ONNX                 u = dout w silu(z),  n = rsqrt(mean(y^2) + eps),
//                        dy = n (u - y n^2 mean(u y)),  dz = dout w y n s',
//                        dw += dout y n silu(z)
// The mean is taken off before squares are summed (two reductions), so a row
// whose mean is far from zero loses nothing.
//
// Of the measured copy rate: layer norm 66 % (rows of 1024) to 93 % (16384 x 3840 bf16 46
// us, 81 %), its gradients 48 to 75 % (89 us, 62 %), the gated norm's 72 to 82 % (16384 x
// 4800 bf16 in groups of 100 155 us, 16384 x 4096 f16 in groups of 128 121 us).  The
// gradients are bound by their instructions (24 to 53 an element, the sums over a group
// among them) at 15 or 16 warps an SM: a thread keeps its columns' sums and weights
// besides a row's values, so that no more CTAs fit.
#pragma once

#include <type_traits>

#include "ggrn_mixer.cuh"
#include "ggrn_optin.h"

namespace ggrn {
namespace norms {

enum Kind : int { kLayerNorm = 0, kLayerNormGrad = 1, kMamba2Grad = 2, kOnnxGrad = 3 };

constexpr int kMaxThreads = 768;
constexpr int kAnyThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;

struct Params {
  const void *dout, *x, *gate, *w;
  const float* b;
  void *out, *dgate;
  float *dw, *db;   // [sums, weight columns] each; db may be NULL
  int64_t rows, groups, gs;
  int64_t ds, xs, gts, os, dgs;  // row strides
  int lanes;        // threads of a group's team: a power of two up to 32, or the CTA
  int team_groups;  // groups that the CTA's teams hold at a time
  int team_rows;    // rows that they hold at a time
  int nvec;         // vectors of a group
  float eps, gs_f, inv_gs;  // inv_gs: 1 / gs
};

// How a call is laid out (norms::plan).
struct Plan {
  int elems = 1;     // elements of a vector
  int vpl = 1;       // vectors of a thread (0: the form that reads a group again)
  int threads = 0, lanes = 0, team_groups = 1, team_rows = 1, nvec = 0;
  int64_t slices = 0, blocks = 1;  // grid: rows, groups
  int smem = 0;
  int64_t sums = 0, columns = 0;   // partial sums
};

// E consecutive elements of T.
template <typename T, int E>
struct Block {
  static constexpr int kBytes = E * sizeof(T);
  using Word = typename std::conditional<
      E == 1, T, typename std::conditional<kBytes == 16, uint4, uint2>::type>::type;
  Word w;
  // An asynchronous copy into shared memory, for the thread that starts it only
  // (2 bytes: a plain one).
  __device__ __forceinline__ static void copy(Word* to, const T* from) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (kBytes == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    } else if constexpr (kBytes == 8) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
    } else if constexpr (kBytes == 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
    } else {
      *to = *from;
    }
  }
  // As pairs (one element: the first half of one, the other 0).
  static constexpr int N = E > 1 ? E / 2 : 1;
  __device__ __forceinline__ void get(Two (&v)[N]) const {
    if constexpr (E == 1) {
      v[0] = join(static_cast<float>(w), 0.0f);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = join(__uint_as_float(w.x), __uint_as_float(w.y));
      if constexpr (E == 4) v[1] = join(__uint_as_float(w.z), __uint_as_float(w.w));
    } else {
      v[0] = two(w.x), v[1] = two(w.y);
      if constexpr (E == 8) v[2] = two(w.z), v[3] = two(w.w);
    }
  }
  __device__ __forceinline__ static Two two(uint32_t u) {
    float x, y;
    Elem<T>::unpack2(u, x, y);
    return join(x, y);
  }
  __device__ __forceinline__ static void put(T* p, const Two (&v)[N]) {
    float f[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) split(v[k], f[2 * k], f[2 * k + 1]);
    if constexpr (E == 1) {
      Elem<T>::store1(p, 0, f[0]);
    } else if constexpr (E == Elem<T>::E) {
      st_stream(p, Elem<T>::pack(f));
    } else if constexpr (sizeof(T) == 4) {
      __stcs(reinterpret_cast<float2*>(p), make_float2(f[0], f[1]));
    } else {
      __stcs(reinterpret_cast<uint2*>(p),
             make_uint2(Elem<T>::pack2(f[0], f[1]), Elem<T>::pack2(f[2], f[3])));
    }
  }
};
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
constexpr int kRingMost = 200 << 10;  // bytes of a CTA's ring
// Rows of a ring: those ahead of the one that is read are in flight.
__host__ __device__ constexpr int depth_of(int kind) {
  return kind == kLayerNorm || kind == kLayerNormGrad ? 5 : 4;
}
// Waits until all but the newest `depth` - 1 rows' copies have landed.
template <int DEPTH>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
}
__device__ __forceinline__ void copies_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ Two both(float v) { return join(v, v); }
// A sum kept in two halves (of single elements: in the first).
template <int E>
__device__ __forceinline__ float value(Two s) {
  float x, y;
  split(s, x, y);
  return E == 1 ? x : x + y;
}

// sigmoid(z), as silu<T> has it.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (Elem<T>::kExactSilu) return 1.0f / (1.0f + expf(-z));
  return rcp_approx(1.0f + ex2_approx(z * -1.4426950408889634f));
}

template <typename T>
__device__ __forceinline__ Two sigmoid2(Two z, Two log2e, Two one) {
  if constexpr (Elem<T>::kExactSilu) return each(z, sigmoid<T>);
  return each(add(each(mul(z, log2e), ex2_approx), one), rcp_approx);
}

// The sums of N values over a team, in every one of its threads.  A team that is
// the CTA goes through shared memory, in one of two places in turn (`place`): a
// barrier lies between two uses of a place.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int lanes, float4* s_sum, int place) {
  if (lanes < 32) {
    for (int o = lanes >> 1; o; o >>= 1) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    return;
  }
  // [sum][warp]: read four warps at a time, the places behind the last one zeros
  float* s = reinterpret_cast<float*>(s_sum + place * 3 * (kMaxWarps / 4));
  if (N == 3 && lanes > 32) {
    // three sums in six shuffles: a quarter of the lanes ends with each (and one with
    // nothing)
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, right = lane & 8;
    float a = up ? v[N - 1] : v[0], b = up ? 0.0f : v[1 % N];
    a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[N - 1], 16);
    b += __shfl_xor_sync(0xffffffffu, up ? v[1 % N] : 0.0f, 16);
    float c = right ? b : a;
    c += __shfl_xor_sync(0xffffffffu, right ? a : b, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    // lanes 0, 8, 16: sums 0, 1, 2
    if ((lane & 7) == 0 && lane < 24) s[(lane >> 3) * kMaxWarps + (threadIdx.x >> 5)] = c;
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    if (lanes == 32) return;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) s[k * kMaxWarps + (threadIdx.x >> 5)] = v[k];
    }
  }
  __syncthreads();
  const ulonglong2* q = reinterpret_cast<const ulonglong2*>(s);
  constexpr int F = kMaxWarps / 4;  // reads of a sum
  static_assert(F == 6, "those below");
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const auto four = [&](int i) { return add(q[k * F + i].x, q[k * F + i].y); };
    Two t = four(0);
    if (lanes > 128) t = add(t, four(1));
    if (lanes > 256) t = add(t, add(four(2), four(3)));
    if (lanes > 512) t = add(t, add(four(4), four(5)));
    float x, y;
    split(t, x, y);
    v[k] = x + y;
  }
}
__device__ __forceinline__ void clear_sums(float4* s_sum) {
  for (int i = threadIdx.x; i < 2 * 3 * (kMaxWarps / 4); i += blockDim.x)
    s_sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
}

// s / gs as the forward pass of the gated norm divides, rounded once: a mean of equal
// values is that value, and a gradient has the statistics of its forward pass.  One step
// of Markstein's correction (IBM J. Res. Dev. 34, 1990): q = s (1 / gs) is within 1.5 ulp,
// s - q gs is exact, and q + (s - q gs) (1 / gs) misses the quotient by 2^-23 ulp before
// it is rounded, where a quotient by gs < 2^20 keeps 2^-21 from every midpoint.  (An
// infinite quotient has no remainder.)  The division's own instructions cost 2 to 3 % of the
// gradients' time.
__device__ __forceinline__ float mean_of(float s, const Params& p) {
  const float q = s * p.inv_gs, t = fmaf(fmaf(-q, p.gs_f, s), p.inv_gs, q);
  return fabsf(q) < INFINITY ? t : q;
}

// The weight of element j of a group (column c of the row), widened.
template <int KIND, typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t c, int64_t j) {
  if constexpr (KIND == kOnnxGrad) return Elem<T>::load1(w, j);
  return __ldg(static_cast<const float*>(w) + c);
}

// Matrices that a kind reads.
constexpr int inputs_of(int kind) { return kind == kLayerNorm ? 1 : kind == kLayerNormGrad ? 2 : 3; }

// Threads of an SM that a kernel's registers leave room for, by the elements that a
// thread holds of each matrix, and the most of a CTA.
// (Eight elements: the gated norm's gradients of 16384 x 4800 in groups of 100 take 155 us
// with 96 registers, 16 warps an SM and nothing spilled, and 182 with 80, 24 warps and
// spills.  Elsewhere kernels of the gradients do spill: single elements by four a thread
// 40 to 132 bytes, 16 elements up to 116, 32 elements 640 to 750; not measured apart.)
__host__ __device__ constexpr int room_of(int kind, int elems) {
  return kind == kLayerNorm ? (elems <= 8 ? 1024 : elems <= 16 ? 768 : 512)
                            : (elems <= 4 ? 1024 : elems <= 8 ? 640 : 512);
}
__host__ __device__ constexpr int threads_of(int kind, int elems) {
  return room_of(kind, elems) == 1024 ? 512 : room_of(kind, elems);
}
// Most elements of a thread of a team, and of a CTA that is one.  (A larger group is
// held all the same where a CTA can, with what that spills.)
__host__ __device__ constexpr int team_elems(int kind) { return kind == kLayerNorm ? 32 : 8; }
__host__ __device__ constexpr int cta_elems(int kind) { return kind == kLayerNorm ? 32 : 16; }

// A team goes down its rows; each thread copies its own vectors of the rows
// ahead into its own places of a ring in shared memory (so that no thread waits
// for another's copies), and reads them from there for each pass.
template <int KIND, typename T, int E, int VPL>
__global__ void __launch_bounds__(threads_of(KIND, VPL * E),
                                  room_of(KIND, VPL * E) / threads_of(KIND, VPL * E))
    k_norm(const Params p) {
  constexpr bool kGrad = KIND != kLayerNorm, kGated = KIND == kMamba2Grad || KIND == kOnnxGrad;
  constexpr bool kLayer = !kGated;
  constexpr int M = inputs_of(KIND), kDepth = depth_of(KIND);
  using Vec = Block<T, E>;
  extern __shared__ uint4 s_ring[];
  __shared__ float4 s_sum[2 * 3 * (kMaxWarps / 4)];
  pdl_wait();
  pdl_launch_dependents();
  const int team = threadIdx.x / p.lanes, lane = threadIdx.x - team * p.lanes;
  const int row_of_team = team / p.team_groups;
  const int64_t g = static_cast<int64_t>(blockIdx.y) * p.team_groups + team % p.team_groups;
  const bool mine = row_of_team < p.team_rows && g < p.groups;
  const int64_t c0 = g * p.gs + lane * E;
  const int apart = p.lanes * E;  // elements between a thread's vectors

  const T* x = static_cast<const T*>(p.x) + c0;
  const T* dout = static_cast<const T*>(p.dout) + c0;
  const T* gate = static_cast<const T*>(p.gate) + c0;
  // the thread's places: [row of the ring][M][VPL], a CTA's threads beside each other
  using Word = typename Vec::Word;
  Word* const ring = reinterpret_cast<Word*>(s_ring) + threadIdx.x;
  const int place = M * VPL * blockDim.x;  // of a row
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.team_rows;
  // the thread's vectors: the first `count` of VPL
  int count = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) count += mine && lane + i * p.lanes < p.nvec;
  const auto has = [&](int i) { return i < count; };
  int64_t row = static_cast<int64_t>(blockIdx.x) * p.team_rows + row_of_team, ahead = row;
  x += row * p.xs, dout += row * p.ds, gate += row * p.gts;
  Word* to = ring;
  const auto fetch = [&]() {
    if (ahead < p.rows) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!has(i)) continue;
        Vec::copy(to + i * blockDim.x, x + i * apart);
        if constexpr (kGrad) Vec::copy(to + (VPL + i) * blockDim.x, dout + i * apart);
        if constexpr (kGated) Vec::copy(to + (2 * VPL + i) * blockDim.x, gate + i * apart);
      }
    }
    copies_commit();
    ahead += step;
    x += step * p.xs;
    if constexpr (kGrad) dout += step * p.ds;
    if constexpr (kGated) gate += step * p.gts;
    to = to == ring + (kDepth - 1) * place ? ring : to + place;
  };
  // (vectors behind the group's last one read zeros)
  for (int k = 0; k < kDepth * M; ++k) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!has(i)) ring[(k * VPL + i) * blockDim.x] = Word{};
  }
  for (int k = 0; k < kDepth - 1; ++k) fetch();

  constexpr int N = Vec::N;
  Two w[VPL][N], b[kLayer && !kGrad ? VPL : 1][N];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    float wf[2 * N], bf[2 * N];
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) {
      const int64_t at = i * apart + k;
      const bool in = has(i) && k < E;
      wf[k] = in ? weight_at<KIND, T>(p.w, c0 + at, lane * E + at) : 0.0f;
      if constexpr (kLayer && !kGrad) bf[k] = in && p.b ? __ldg(p.b + c0 + at) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      w[i][k] = join(wf[2 * k], wf[2 * k + 1]);
      if constexpr (kLayer && !kGrad) b[i][k] = join(bf[2 * k], bf[2 * k + 1]);
      // (kept, not loaded again for every row)
      asm volatile("" : "+l"(w[i][k]));
      if constexpr (kLayer && !kGrad) asm volatile("" : "+l"(b[i][k]));
    }
  }
  Two dw[kGrad ? VPL : 1][N], db[KIND == kLayerNormGrad ? VPL : 1][N];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (kGrad) dw[i][k] = 0;
      if constexpr (KIND == kLayerNormGrad) db[i][k] = 0;
    }
  }
  const Two one = held(1.0f), minus = held(-1.0f), log2e = held(-1.4426950408889634f);
  if (p.lanes > 32) clear_sums(s_sum);

  int turn = 0;
  const Word* from = ring;
  T* out = static_cast<T*>(p.out) + row * p.os + c0;
  T* dgate = static_cast<T*>(p.dgate) + row * p.dgs + c0;
  // (the rows of the CTA's teams follow each other: all take as many turns)
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.team_rows; first < p.rows;
       first += step) {
    fetch();
    copies_wait<kDepth>();
    // (a team without a group has n = inf of its zeros where eps is 0)
    const bool live = mine && row < p.rows;
    const auto load = [&](int m, int i, Two (&f)[N]) {
      Vec v;
      v.w = from[(m * VPL + i) * blockDim.x];
      v.get(f);
    };
    if constexpr (kLayer) {
      Two x[VPL][N], g[kGrad ? VPL : 1][N];
      Two sum = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        load(0, i, x[i]);
        if constexpr (kGrad) load(1, i, g[i]);
#pragma unroll
        for (int k = 0; k < N; ++k) sum = add(sum, x[i][k]);
      }
      float mean[1] = {value<E>(sum)};
      team_sum<1>(mean, p.lanes, s_sum, 0);
      // (divided: of a row of one value nothing is left)
      const Two less = both(-mean_of(mean[0], p));
      constexpr int S = kGrad ? 3 : 1;
      Two q[3] = {0, 0, 0};
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const Two by = has(i) ? less : 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          x[i][k] = add(x[i][k], by);
          q[0] = fma(x[i][k], x[i][k], q[0]);
          if constexpr (kGrad) {
            const Two u = mul(g[i][k], w[i][k]);
            q[1] = add(q[1], u);
            q[2] = fma(u, x[i][k], q[2]);
          }
        }
      }
      float s[S];
#pragma unroll
      for (int k = 0; k < S; ++k) s[k] = value<E>(q[k]);
      team_sum<S>(s, p.lanes, s_sum, 1);
      const float nf = rsqrtf(mean_of(s[0], p) + p.eps);
      const Two n = both(nf);
      if (live) {
        Two mu = 0, mud = 0;
        if constexpr (kGrad) {
          mu = both(-s[1] * p.inv_gs);
          mud = both(-s[2] * p.inv_gs * nf * nf);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          Two o[N];
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const Two xh = mul(x[i][k], n);
            if constexpr (kGrad) {
              o[k] = mul(fma(x[i][k], mud, fma(g[i][k], w[i][k], mu)), n);
              dw[i][k] = fma(g[i][k], xh, dw[i][k]);
              db[i][k] = add(g[i][k], db[i][k]);
            } else {
              o[k] = fma(xh, w[i][k], b[i][k]);
            }
          }
          if (has(i)) Vec::put(out + i * apart, o);
        }
      }
    } else {
      // MAMBA2 keeps silu, y s', y silu and dout; ONNX u, dout w s', y and dout silu
      Two ka[VPL][N], kb[VPL][N], kv[VPL][N], kg[VPL][N];
      Two q[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        Two y[N], g[N], z[N];
        load(0, i, y), load(1, i, g), load(2, i, z);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const Two sig = sigmoid2<T>(z[k], log2e, one);
          const Two act = mul(z[k], sig);
          const Two slope = mul(fma(z[k], fma(sig, minus, one), one), sig);
          const Two u = mul(g[k], w[i][k]);
          if constexpr (KIND == kMamba2Grad) {
            ka[i][k] = act;
            kb[i][k] = mul(y[k], slope);
            kv[i][k] = mul(y[k], act);
            kg[i][k] = g[k];
            q[1] = fma(u, kv[i][k], q[1]);
          } else {
            ka[i][k] = mul(u, act);
            kb[i][k] = mul(u, slope);
            kv[i][k] = y[k];
            kg[i][k] = mul(g[k], act);
            q[1] = fma(ka[i][k], y[k], q[1]);
          }
          q[0] = fma(kv[i][k], kv[i][k], q[0]);
        }
      }
      float s[2] = {value<E>(q[0]), value<E>(q[1])};
      team_sum<2>(s, p.lanes, s_sum, turn++ & 1);
      const float nf = rsqrtf(mean_of(s[0], p) + p.eps);
      const Two n = both(nf), muv = both(-s[1] * p.inv_gs * nf * nf);
      if (live) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          Two dy[N], dz[N];
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const Two vn = mul(kv[i][k], n);
            dw[i][k] = fma(kg[i][k], vn, dw[i][k]);
            if constexpr (KIND == kMamba2Grad) {
              const Two dv = mul(fma(kv[i][k], muv, mul(kg[i][k], w[i][k])), n);
              dy[k] = mul(dv, ka[i][k]);
              dz[k] = mul(dv, kb[i][k]);
            } else {
              dy[k] = mul(fma(kv[i][k], muv, ka[i][k]), n);
              dz[k] = mul(kb[i][k], vn);
            }
          }
          if (has(i)) {
            Vec::put(out + i * apart, dy);
            Vec::put(dgate + i * apart, dz);
          }
        }
      }
      dgate += step * p.dgs;
    }
    out += step * p.os;
    row += step;
    from = from == ring + (kDepth - 1) * place ? ring : from + place;
  }

  if constexpr (kGrad) {
    // The CTA's sums: teams on other rows of a group (ONNX: all teams) in order.
    const int teams = KIND == kOnnxGrad ? p.team_rows * p.team_groups : p.team_rows;
    const int next = KIND == kOnnxGrad ? 1 : p.team_groups;  // teams of the same columns
    const bool writes = mine && (KIND == kOnnxGrad ? team == 0 : row_of_team == 0);
    const int64_t columns = KIND == kOnnxGrad ? p.gs : p.groups * p.gs;
    const int64_t sum = KIND == kOnnxGrad ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x;
    const int64_t col0 = KIND == kOnnxGrad ? lane * E : c0;
    float* s_acc = reinterpret_cast<float*>(s_ring);  // (the ring is at its end)
    copies_wait_all();
    const auto finish = [&](const Two (&sums)[VPL][N], float* out) {
      float a[VPL][2 * N];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int k = 0; k < N; ++k) split(sums[i][k], a[i][2 * k], a[i][2 * k + 1]);
      }
      if (teams > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
#pragma unroll
          for (int k = 0; k < E; ++k) s_acc[(i * E + k) * blockDim.x + threadIdx.x] = a[i][k];
        }
        __syncthreads();
        if (writes) {
          for (int t = 1; t < teams; ++t) {
            const int other = threadIdx.x + t * next * p.lanes;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
#pragma unroll
              for (int k = 0; k < E; ++k) a[i][k] += s_acc[(i * E + k) * blockDim.x + other];
            }
          }
        }
      }
      if (!writes) return;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!has(i)) continue;
#pragma unroll
        for (int k = 0; k < E; ++k) out[sum * columns + col0 + i * apart + k] = a[i][k];
      }
    };
    finish(dw, p.dw);
    if constexpr (KIND == kLayerNormGrad) {
      if (p.db) finish(db, p.db);
    }
  }
}

// Any layout and any group: a CTA for each group of its rows, which it reads
// again for every pass (from L1 and L2).  For what the threads of a CTA, or its ring of
// rows in shared memory, do not hold: more than 2048 single elements, layer norm beyond
// 16384 columns (f32: 10240), its gradients beyond 10240 (5120), groups of the gated
// norm beyond 8192 (4096).  Each thread owns the same columns in every row; their sums
// lie in its CTA's row of the partial sums.  Three passes, and sums read and written for
// each row: the gated norm's gradients of 4096 x 12288 bf16 in one group take 413 us
// (floor 74), of 4096 x 5120 f32 167 (62), layer norm's of 4096 x 7680 f32 209 (56).
template <int KIND, typename T>
__global__ void __launch_bounds__(kAnyThreads) k_norm_any(const Params p) {
  constexpr bool kGrad = KIND != kLayerNorm, kGated = KIND == kMamba2Grad || KIND == kOnnxGrad;
  __shared__ float4 s_sum[2 * 3 * (kMaxWarps / 4)];
  pdl_wait();
  pdl_launch_dependents();
  clear_sums(s_sum);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * p.gs;
  const int64_t columns = KIND == kOnnxGrad ? p.gs : p.groups * p.gs;
  const int64_t sum = KIND == kOnnxGrad ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x;
  float* dw = p.dw + sum * columns + (KIND == kOnnxGrad ? 0 : c0);
  float* db = p.db + sum * columns;
  bool fresh = true;
  int place = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.xs + c0;
    const T* dout = static_cast<const T*>(p.dout) + row * p.ds + c0;
    const T* gate = static_cast<const T*>(p.gate) + row * p.gts + c0;
    T* out = static_cast<T*>(p.out) + row * p.os + c0;
    float mean = 0.0f;
    if constexpr (!kGated) {
      float m[1] = {0.0f};
      for (int64_t j = threadIdx.x; j < p.gs; j += blockDim.x) m[0] += static_cast<float>(x[j]);
      team_sum<1>(m, blockDim.x, s_sum, place);
      place ^= 1;
      mean = mean_of(m[0], p);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int64_t j = threadIdx.x; j < p.gs; j += blockDim.x) {
      const float wj = kGrad ? weight_at<KIND, T>(p.w, c0 + j, j) : 0.0f;
      float v = static_cast<float>(x[j]) - mean, u = 0.0f;
      if constexpr (kGrad) u = static_cast<float>(dout[j]) * wj;
      if constexpr (kGated) {
        const float z = static_cast<float>(gate[j]), act = z * sigmoid<T>(z);
        if constexpr (KIND == kMamba2Grad) v *= act;
        else u *= act;
      }
      s[0] = fmaf(v, v, s[0]);
      s[1] += u;
      s[2] = fmaf(u, v, s[2]);
    }
    team_sum<3>(s, blockDim.x, s_sum, place);
    place ^= 1;
    const float n = rsqrtf(mean_of(s[0], p) + p.eps);
    const float mu = kGated ? 0.0f : s[1] * p.inv_gs;
    const float muv = s[2] * p.inv_gs * n * n;
    for (int64_t j = threadIdx.x; j < p.gs; j += blockDim.x) {
      const float wj = weight_at<KIND, T>(p.w, c0 + j, j);
      const float d = static_cast<float>(x[j]) - mean;
      if constexpr (!kGrad) {
        Elem<T>::store1(out, j, fmaf(d * n, wj, p.b ? __ldg(p.b + j) : 0.0f));
        continue;
      }
      const float gv = static_cast<float>(dout[j]);
      float add;
      if constexpr (KIND == kLayerNormGrad) {
        Elem<T>::store1(out, j, n * (fmaf(gv, wj, -mu) - d * muv));
        add = gv * (d * n);
        if (p.db) db[j] = fresh ? gv : db[j] + gv;
      } else {
        const float z = static_cast<float>(gate[j]), sg = sigmoid<T>(z), act = z * sg;
        const float slope = sg * fmaf(z, 1.0f - sg, 1.0f);
        float dy, dz;
        if constexpr (KIND == kMamba2Grad) {
          const float v = d * act, dv = n * (gv * wj - v * muv);
          dy = dv * act, dz = dv * d * slope, add = gv * (v * n);
        } else {
          dy = n * (gv * wj * act - d * muv), dz = gv * wj * (d * n) * slope;
          add = gv * act * (d * n);
        }
        Elem<T>::store1(out, j, dy);
        Elem<T>::store1(static_cast<T*>(p.dgate) + row * p.dgs + c0, j, dz);
      }
      dw[j] = fresh ? add : dw[j] + add;
    }
    fresh = false;
  }
}

// ---------------------------------------------------------------------------
// Launch of a plan.
// ---------------------------------------------------------------------------
template <int KIND, typename T, int E, int VPL, typename Go>
int go_with(const Plan& k, Go go) {
  if (k.smem > 40 << 10) {  // (48 KB with what a kernel has by itself)
    const cudaError_t e = allow_shared_memory<k_norm<KIND, T, E, VPL>>(kRingMost);
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return GGRN_ERR_CUDA;
    }
  }
  return go(k_norm<KIND, T, E, VPL>);
}
template <int KIND, typename T, int E, typename Go>
int go_vpl(const Plan& k, Go go) {
  if (k.vpl == 1) return go_with<KIND, T, E, 1>(k, go);
  if (k.vpl == 2) return go_with<KIND, T, E, 2>(k, go);
  return go_with<KIND, T, E, 4>(k, go);
}
template <int KIND, typename T>
int launch_kind(const Params& p, const Plan& k, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(k.slices), static_cast<unsigned>(k.blocks));
  const auto go = [&](auto kernel) {
    return mixer::launch(kernel, grid, static_cast<unsigned>(k.threads), k.smem, s, p);
  };
  if (k.vpl == 0) return go(k_norm_any<KIND, T>);
  constexpr int V = 16 / sizeof(T);
  if (k.elems == V) return go_vpl<KIND, T, V>(k, go);
  if (k.elems == V / 2) return go_vpl<KIND, T, V / 2>(k, go);
  return go_vpl<KIND, T, 1>(k, go);
}

int launch_f32(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_f16(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_bf16(int kind, const Params& p, const Plan& k, cudaStream_t s);

}  // namespace norms
}  // namespace ggrn
