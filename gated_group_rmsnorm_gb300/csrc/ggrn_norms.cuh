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
#pragma once

#include <type_traits>

#include "ggrn_mixer.cuh"
#include "ggrn_optin.h"

namespace ggrn {
namespace norms {

enum Kind : int { kLayerNorm = 0, kLayerNormGrad = 1, kMamba2Grad = 2, kOnnxGrad = 3 };

constexpr int kMaxThreads = 512;
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
  int depth;        // rows of copies in flight
  float eps, gs_f;
};

// How a call is laid out (norms::plan).
struct Plan {
  int elems = 1;     // elements of a vector
  int vpl = 1;       // vectors of a thread (0: the form that reads a group again)
  int threads = 0, lanes = 0, team_groups = 1, team_rows = 1, nvec = 0;
  int64_t slices = 0, blocks = 1;  // grid: rows, groups
  int depth = 1, smem = 0;
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
  __device__ __forceinline__ void get(float (&f)[E]) const {
    if constexpr (E == Elem<T>::E) {
      Elem<T>::unpack(w, f);
    } else if constexpr (E == 1) {
      f[0] = static_cast<float>(w);
    } else if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
    } else {
      Elem<T>::unpack2(w.x, f[0], f[1]);
      Elem<T>::unpack2(w.y, f[2], f[3]);
    }
  }
  __device__ __forceinline__ static void put(T* p, const float (&f)[E]) {
    if constexpr (E == Elem<T>::E) {
      st_stream(p, Elem<T>::pack(f));
    } else if constexpr (E == 1) {
      Elem<T>::store1(p, 0, f[0]);
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
// Waits until at most n of the thread's groups of copies are in flight.
__device__ __forceinline__ void copies_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}
constexpr int kMaxDepth = 4;

// Pairs of f32 (see mul2 and fma2), for an even E; one by one for E = 1.
// d[k] = a[k] b[k] + c[k] with b or c the same for all where it is a number.
template <int E, typename B, typename C>
__device__ __forceinline__ void fma_n(float (&d)[E], const float (&a)[E], const B& b, const C& c) {
  const auto at = [](const auto& v, int k) {
    if constexpr (std::is_same<std::decay_t<decltype(v)>, float>::value) return v;
    else return v[k];
  };
  if constexpr (E == 1) {
    d[0] = fmaf(a[0], at(b, 0), at(c, 0));
  } else {
#pragma unroll
    for (int k = 0; k < E; k += 2)
      fma2(d[k], d[k + 1], a[k], a[k + 1], at(b, k), at(b, k + 1), at(c, k), at(c, k + 1));
  }
}
template <int E, typename B>
__device__ __forceinline__ void mul_n(float (&d)[E], const float (&a)[E], const B& b) {
  const auto at = [](const auto& v, int k) {
    if constexpr (std::is_same<std::decay_t<decltype(v)>, float>::value) return v;
    else return v[k];
  };
  if constexpr (E == 1) {
    d[0] = a[0] * at(b, 0);
  } else {
#pragma unroll
    for (int k = 0; k < E; k += 2)
      mul2(d[k], d[k + 1], a[k], a[k + 1], at(b, k), at(b, k + 1));
  }
}
// A sum kept in two halves.
struct Sum {
  float lo = 0.0f, hi = 0.0f;
  template <int E>
  __device__ __forceinline__ void add(const float (&a)[E]) {
    if constexpr (E == 1) {
      lo += a[0];
    } else {
#pragma unroll
      for (int k = 0; k < E; k += 2) fma2(lo, hi, a[k], a[k + 1], 1.0f, 1.0f, lo, hi);
    }
  }
  template <int E>
  __device__ __forceinline__ void add(const float (&a)[E], const float (&b)[E]) {
    if constexpr (E == 1) {
      lo = fmaf(a[0], b[0], lo);
    } else {
#pragma unroll
      for (int k = 0; k < E; k += 2) fma2(lo, hi, a[k], a[k + 1], b[k], b[k + 1], lo, hi);
    }
  }
  __device__ __forceinline__ float value() const { return lo + hi; }
};

// sigmoid(z), as silu<T> has it.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (Elem<T>::kExactSilu) return 1.0f / (1.0f + expf(-z));
  return rcp_approx(1.0f + ex2_approx(z * -1.4426950408889634f));
}

// The sums of N values over a team, in every one of its threads.  A team that is
// the CTA goes through shared memory, in one of two places in turn (`place`): a
// barrier lies between two uses of a place.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int lanes, float4* s_sum, int place) {
  const int most = lanes < 32 ? lanes : 32;
  for (int o = most >> 1; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (lanes <= 32) return;
  // [sum][warp]: read four warps at a time, the places behind the last one zeros
  float* s = reinterpret_cast<float*>(s_sum + place * 3 * (kMaxWarps / 4));
  const int warp = threadIdx.x >> 5, fours = (lanes + 127) >> 7;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k * kMaxWarps + warp] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float4* q = reinterpret_cast<const float4*>(s + k * kMaxWarps);
    v[k] = 0.0f;
    for (int w = 0; w < fours; ++w) v[k] += (q[w].x + q[w].y) + (q[w].z + q[w].w);
  }
}
__device__ __forceinline__ void clear_sums(float4* s_sum) {
  for (int i = threadIdx.x; i < 2 * 3 * (kMaxWarps / 4); i += blockDim.x)
    s_sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
}

// The weight of element j of a group (column c of the row), widened.
template <int KIND, typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t c, int64_t j) {
  if constexpr (KIND == kOnnxGrad) return Elem<T>::load1(w, j);
  return __ldg(static_cast<const float*>(w) + c);
}

// Matrices that a kind reads.
constexpr int inputs_of(int kind) { return kind == kLayerNorm ? 1 : kind == kLayerNormGrad ? 2 : 3; }

// Most threads of a CTA, and CTAs that the registers have to leave room for.
constexpr int threads_of(int vpl) { return vpl == 4 ? kMaxThreads : 256; }
constexpr int resident_of(int vpl) { return vpl == 1 ? 4 : vpl == 2 ? 3 : 1; }

// A team goes down its rows; each thread copies its own vectors of the rows
// ahead into its own places of a ring in shared memory (so that no thread waits
// for another's copies), and reads them from there for each pass.
template <int KIND, typename T, int E, int VPL>
__global__ void __launch_bounds__(threads_of(VPL), resident_of(VPL)) k_norm(const Params p) {
  constexpr bool kGrad = KIND != kLayerNorm, kGated = KIND == kMamba2Grad || KIND == kOnnxGrad;
  constexpr bool kLayer = !kGated;
  constexpr int M = inputs_of(KIND);
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
  // the thread's places: [depth][M][VPL], a CTA's threads beside each other
  using Word = typename Vec::Word;
  Word* const ring = reinterpret_cast<Word*>(s_ring) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.team_rows;
  const auto has = [&](int i) { return lane + i * p.lanes < p.nvec; };
  const auto fetch = [&](int64_t row, int place) {
    if (mine && row < p.rows) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!has(i)) continue;
        Word* to = ring + (place * M * VPL + i) * blockDim.x;
        Vec::copy(to, x + row * p.xs + i * apart);
        if constexpr (kGrad) Vec::copy(to + VPL * blockDim.x, dout + row * p.ds + i * apart);
        if constexpr (kGated) Vec::copy(to + 2 * VPL * blockDim.x, gate + row * p.gts + i * apart);
      }
    }
    copies_commit();
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * p.team_rows + row_of_team;
  for (int k = 0; k < p.depth - 1; ++k) fetch(row + k * step, k);

  float w[VPL][E], b[kLayer && !kGrad ? VPL : 1][E];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int64_t at = i * apart + k;
      w[i][k] = mine && has(i) ? weight_at<KIND, T>(p.w, c0 + at, lane * E + at) : 0.0f;
      if constexpr (kLayer && !kGrad) b[i][k] = mine && has(i) && p.b ? __ldg(p.b + c0 + at) : 0.0f;
    }
  }
  float dw[kGrad ? VPL : 1][E], db[KIND == kLayerNormGrad ? VPL : 1][E];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      if constexpr (kGrad) dw[i][k] = 0.0f;
      if constexpr (KIND == kLayerNormGrad) db[i][k] = 0.0f;
    }
  }
  if (p.lanes > 32) clear_sums(s_sum);

  int place = 0, turn = 0;
  // (the rows of the CTA's teams follow each other: all take as many turns)
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.team_rows; first < p.rows;
       first += step, row += step) {
    {
      const int ahead = place == 0 ? p.depth - 1 : place - 1;
      fetch(row + (p.depth - 1) * step, ahead);
    }
    copies_wait(p.depth - 1);
    const bool live = mine && row < p.rows;
    const Word* from = ring + place * M * VPL * blockDim.x;
    place = place + 1 == p.depth ? 0 : place + 1;
    const auto load = [&](int m, int i, float (&f)[E]) {
      Vec v;
      v.w = from[(m * VPL + i) * blockDim.x];
      v.get(f);
    };

    if constexpr (kLayer) {
      float mean[1];
      {
        Sum s;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!live || !has(i)) continue;
          float f[E];
          load(0, i, f);
          s.add(f);
        }
        mean[0] = s.value();
      }
      team_sum<1>(mean, p.lanes, s_sum, 0);
      const float less = -__fdiv_rn(mean[0], p.gs_f);
      constexpr int S = kGrad ? 3 : 1;
      Sum q[3];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!live || !has(i)) continue;
        float d[E];
        load(0, i, d);
        fma_n(d, d, 1.0f, less);
        q[0].add(d, d);
        if constexpr (kGrad) {
          float u[E];
          load(1, i, u);
          mul_n(u, u, w[i]);
          q[1].add(u);
          q[2].add(u, d);
        }
      }
      float s[S];
#pragma unroll
      for (int k = 0; k < S; ++k) s[k] = q[k].value();
      team_sum<S>(s, p.lanes, s_sum, 1);
      const float n = rsqrtf(__fdiv_rn(s[0], p.gs_f) + p.eps);
      float mu = 0.0f, mud = 0.0f;
      if constexpr (kGrad) {
        mu = -__fdiv_rn(s[1], p.gs_f);
        mud = -__fdiv_rn(s[2], p.gs_f) * n * n;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!live || !has(i)) continue;
        float d[E], o[E];
        load(0, i, d);
        fma_n(d, d, 1.0f, less);
        if constexpr (kGrad) {
          float gv[E];
          load(1, i, gv);
          fma_n(o, gv, w[i], mu);
          float t[E];
          fma_n(t, d, mud, o);
          mul_n(o, t, n);
          mul_n(d, d, n);
          fma_n(dw[i], gv, d, dw[i]);
          fma_n(db[i], gv, 1.0f, db[i]);
        } else {
          mul_n(d, d, n);
          fma_n(o, d, w[i], b[i]);
        }
        Vec::put(static_cast<T*>(p.out) + row * p.os + c0 + i * apart, o);
      }
    } else {
      Sum q[2];
      float sig[VPL][E];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!live || !has(i)) continue;
        float y[E], u[E], z[E];
        load(0, i, y), load(1, i, u), load(2, i, z);
#pragma unroll
        for (int k = 0; k < E; ++k) sig[i][k] = sigmoid<T>(z[k]);
        mul_n(z, z, sig[i]);  // silu
        mul_n(u, u, w[i]);
        if constexpr (KIND == kMamba2Grad) mul_n(y, y, z);
        else mul_n(u, u, z);
        q[0].add(y, y);
        q[1].add(u, y);
      }
      float s[2] = {q[0].value(), q[1].value()};
      team_sum<2>(s, p.lanes, s_sum, turn++ & 1);
      const float n = rsqrtf(__fdiv_rn(s[0], p.gs_f) + p.eps);
      const float muv = -__fdiv_rn(s[1], p.gs_f) * n * n;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!live || !has(i)) continue;
        float y[E], gv[E], z[E], act[E], slope[E], u[E], t[E];
        load(0, i, y), load(1, i, gv), load(2, i, z);
        mul_n(act, z, sig[i]);
        fma_n(t, sig[i], -1.0f, 1.0f);
        fma_n(t, z, t, 1.0f);
        mul_n(slope, t, sig[i]);
        mul_n(u, gv, w[i]);
        if constexpr (KIND == kMamba2Grad) {
          float v[E];
          mul_n(v, y, act);
          fma_n(t, v, muv, u);
          mul_n(t, t, n);  // dv
          mul_n(v, v, n);
          fma_n(dw[i], gv, v, dw[i]);
          mul_n(act, t, act);    // dy
          mul_n(t, t, y);
          mul_n(slope, t, slope);  // dz
        } else {
          mul_n(t, u, act);
          fma_n(t, y, muv, t);
          mul_n(y, y, n);
          mul_n(gv, gv, act);
          fma_n(dw[i], gv, y, dw[i]);
          mul_n(act, t, n);      // dy
          mul_n(u, u, y);
          mul_n(slope, u, slope);  // dz
        }
        Vec::put(static_cast<T*>(p.out) + row * p.os + c0 + i * apart, act);
        Vec::put(static_cast<T*>(p.dgate) + row * p.dgs + c0 + i * apart, slope);
      }
    }
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
    copies_wait(0);
    const auto finish = [&](float (&a)[VPL][E], float* out) {
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
// again for every pass (from L1 and L2).  Each thread owns the same columns in
// every row; their sums lie in its CTA's row of the partial sums.
template <int KIND, typename T>
__global__ void __launch_bounds__(kMaxThreads) k_norm_any(const Params p) {
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
      mean = __fdiv_rn(m[0], p.gs_f);
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
    const float n = rsqrtf(__fdiv_rn(s[0], p.gs_f) + p.eps);
    const float mu = kGated ? 0.0f : __fdiv_rn(s[1], p.gs_f);
    const float muv = __fdiv_rn(s[2], p.gs_f) * n * n;
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
template <int KIND, typename T, int E, typename Go>
int go_vpl(const Params& p, const Plan& k, Go go) {
  constexpr int kMost = 200 << 10;
  if (k.smem > 40 << 10) {  // (48 KB with what a kernel has by itself)
    cudaError_t e = k.vpl == 1   ? allow_shared_memory<k_norm<KIND, T, E, 1>>(kMost)
                    : k.vpl == 2 ? allow_shared_memory<k_norm<KIND, T, E, 2>>(kMost)
                                 : allow_shared_memory<k_norm<KIND, T, E, 4>>(kMost);
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return GGRN_ERR_CUDA;
    }
  }
  if (k.vpl == 1) return go(k_norm<KIND, T, E, 1>);
  if (k.vpl == 2) return go(k_norm<KIND, T, E, 2>);
  return go(k_norm<KIND, T, E, 4>);
}
template <int KIND, typename T>
int launch_kind(const Params& p, const Plan& k, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(k.slices), static_cast<unsigned>(k.blocks));
  const auto go = [&](auto kernel) {
    return mixer::launch(kernel, grid, static_cast<unsigned>(k.threads), k.smem, s, p);
  };
  if (k.vpl == 0) return go(k_norm_any<KIND, T>);
  constexpr int V = 16 / sizeof(T);
  if (k.elems == V) return go_vpl<KIND, T, V>(p, k, go);
  if (k.elems == V / 2) return go_vpl<KIND, T, V / 2>(p, k, go);
  return go_vpl<KIND, T, 1>(p, k, go);
}

int launch_f32(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_f16(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_bf16(int kind, const Params& p, const Plan& k, cudaStream_t s);

}  // namespace norms
}  // namespace ggrn
