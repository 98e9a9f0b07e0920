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

namespace ggrn {
namespace norms {

enum Kind : int { kLayerNorm = 0, kLayerNormGrad = 1, kMamba2Grad = 2, kOnnxGrad = 3 };

constexpr int kMaxThreads = 512;

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
  float eps, gs_f;
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
  using Word = typename std::conditional<
      E == 1, T,
      typename std::conditional<E * sizeof(T) == 16, uint4, uint2>::type>::type;
  Word w;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (E * sizeof(T) == 16) {
      w = ld_stream(p);
    } else if constexpr (E > 1) {
      w = __ldcs(reinterpret_cast<const uint2*>(p));
    } else {
      w = *p;
    }
  }
  __device__ __forceinline__ void clear() {
    if constexpr (E > 1) {
      w = Word{};
    } else {
      Elem<T>::store1(&w, 0, 0.0f);
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
__device__ __forceinline__ void team_sum(float (&v)[N], int lanes, float* s_sum, int place) {
  const int most = lanes < 32 ? lanes : 32;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (o < most) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
  }
  if (lanes <= 32) return;
  constexpr int kWarps = kMaxThreads / 32;
  float* s = s_sum + place * kWarps * 8;
  const int warp = threadIdx.x >> 5, warps = lanes >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[warp * N + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.0f;
  for (int w = 0; w < warps; ++w) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += s[w * N + k];
  }
}

// Rows of a team in flight.
constexpr int rows_ahead(int elem_bytes, int elems, int vpl) {
  return vpl == 1 ? (elem_bytes * elems == 16 ? 2 : 4) : 1;
}

// The weight of element j of a group (column c of the row), widened.
template <int KIND, typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t c, int64_t j) {
  if constexpr (KIND == kOnnxGrad) return Elem<T>::load1(w, j);
  return __ldg(static_cast<const float*>(w) + c);
}

// One group (VPL vectors of E elements a thread) of each of RB rows.
template <int KIND, typename T, int E, int VPL, int RB>
__global__ void __launch_bounds__(kMaxThreads, VPL == 1 ? 2 : 1) k_norm(const Params p) {
  constexpr bool kGrad = KIND != kLayerNorm, kGated = KIND == kMamba2Grad || KIND == kOnnxGrad;
  constexpr bool kLayer = !kGated;
  extern __shared__ float s_acc[];
  __shared__ float s_sum[2 * (kMaxThreads / 32) * 8];
  pdl_wait();
  pdl_launch_dependents();
  const int team = threadIdx.x / p.lanes, lane = threadIdx.x - team * p.lanes;
  const int row_of_team = team / p.team_groups;
  const int64_t g = static_cast<int64_t>(blockIdx.y) * p.team_groups + team % p.team_groups;
  const bool mine = row_of_team < p.team_rows && g < p.groups;
  const int64_t c0 = g * p.gs;

  bool has[VPL];
  float w[VPL][E], b[kLayer && !kGrad ? VPL : 1][E];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int v = lane + i * p.lanes;
    has[i] = mine && v < p.nvec;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      w[i][k] = has[i] ? weight_at<KIND, T>(p.w, c0 + v * E + k, v * E + k) : 0.0f;
      if constexpr (kLayer && !kGrad)
        b[i][k] = has[i] && p.b ? __ldg(p.b + v * E + k) : 0.0f;
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

  const T* x = static_cast<const T*>(p.x) + c0;
  const T* dout = static_cast<const T*>(p.dout) + c0;
  const T* gate = static_cast<const T*>(p.gate) + c0;
  Block<T, E> xr[RB][VPL], gr[kGrad ? RB : 1][VPL], zr[kGated ? RB : 1][VPL];
  auto fetch = [&](int64_t row0) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int64_t row = row0 + r * p.team_rows + row_of_team;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int64_t at = (lane + i * p.lanes) * E;
        if (has[i] && row < p.rows) {
          xr[r][i].load(x + row * p.xs + at);
          if constexpr (kGrad) gr[r][i].load(dout + row * p.ds + at);
          if constexpr (kGated) zr[r][i].load(gate + row * p.gts + at);
        } else {
          xr[r][i].clear();
          if constexpr (kGrad) gr[r][i].clear();
          if constexpr (kGated) zr[r][i].clear();
        }
      }
    }
  };

  const int64_t turn_rows = static_cast<int64_t>(p.team_rows) * RB;
  int place = 0;
  int64_t row0 = blockIdx.x * turn_rows;
  fetch(row0);
  for (; row0 < p.rows; row0 += gridDim.x * turn_rows) {
    Block<T, E> xc[RB][VPL], gc[kGrad ? RB : 1][VPL], zc[kGated ? RB : 1][VPL];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        xc[r][i] = xr[r][i];
        if constexpr (kGrad) gc[r][i] = gr[r][i];
        if constexpr (kGated) zc[r][i] = zr[r][i];
      }
    }
    if (row0 + gridDim.x * turn_rows < p.rows) fetch(row0 + gridDim.x * turn_rows);

    if constexpr (kLayer) {
      float mean[RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        mean[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          float f[E];
          xc[r][i].get(f);
#pragma unroll
          for (int k = 0; k < E; ++k) mean[r] += f[k];
        }
      }
      team_sum<RB>(mean, p.lanes, s_sum, 0);
      constexpr int S = kGrad ? 3 : 1;
      float s[S * RB];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        mean[r] = __fdiv_rn(mean[r], p.gs_f);
#pragma unroll
        for (int q = 0; q < S; ++q) s[S * r + q] = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!has[i]) continue;
          float f[E], gv[E];
          xc[r][i].get(f);
          if constexpr (kGrad) gc[r][i].get(gv);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float d = f[k] - mean[r];
            s[S * r] = fmaf(d, d, s[S * r]);
            if constexpr (kGrad) {
              const float u = gv[k] * w[i][k];
              s[S * r + 1] += u;
              s[S * r + 2] = fmaf(u, d, s[S * r + 2]);
            }
          }
        }
      }
      if constexpr (S * RB <= 8) {
        team_sum<S * RB>(s, p.lanes, s_sum, 1);
      } else {  // (places hold eight sums of a warp)
        static_assert(S * RB <= 8 || RB == 4, "rows in two halves");
        float s0[S * 2], s1[S * 2];
#pragma unroll
        for (int k = 0; k < S * 2; ++k) s0[k] = s[k], s1[k] = s[S * 2 + k];
        team_sum<S * 2>(s0, p.lanes, s_sum, 1);
        if (p.lanes > 32) __syncthreads();
        team_sum<S * 2>(s1, p.lanes, s_sum, 1);
#pragma unroll
        for (int k = 0; k < S * 2; ++k) s[k] = s0[k], s[S * 2 + k] = s1[k];
      }
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int64_t row = row0 + r * p.team_rows + row_of_team;
        const float n = rsqrtf(__fdiv_rn(s[S * r], p.gs_f) + p.eps);
        float mu = 0.0f, mud = 0.0f;
        if constexpr (kGrad) {
          mu = __fdiv_rn(s[S * r + 1], p.gs_f);
          mud = __fdiv_rn(s[S * r + 2], p.gs_f) * n * n;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!has[i] || row >= p.rows) continue;
          float f[E], gv[E], o[E];
          xc[r][i].get(f);
          if constexpr (kGrad) gc[r][i].get(gv);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float d = f[k] - mean[r];
            if constexpr (kGrad) {
              o[k] = n * (fmaf(gv[k], w[i][k], -mu) - d * mud);
              dw[i][k] = fmaf(gv[k], d * n, dw[i][k]);
              db[i][k] += gv[k];
            } else {
              o[k] = fmaf(d * n, w[i][k], b[i][k]);
            }
          }
          Block<T, E>::put(static_cast<T*>(p.out) + row * p.os + c0 + (lane + i * p.lanes) * E, o);
        }
      }
    } else {
      float s[2 * RB], sig[RB][VPL][E];
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        s[2 * r] = s[2 * r + 1] = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          float y[E], gv[E], z[E];
          xc[r][i].get(y), gc[r][i].get(gv), zc[r][i].get(z);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            sig[r][i][k] = sigmoid<T>(z[k]);
            const float act = z[k] * sig[r][i][k];
            const float v = KIND == kMamba2Grad ? y[k] * act : y[k];
            const float u = KIND == kMamba2Grad ? gv[k] * w[i][k] : gv[k] * w[i][k] * act;
            if (has[i]) {
              s[2 * r] = fmaf(v, v, s[2 * r]);
              s[2 * r + 1] = fmaf(u, v, s[2 * r + 1]);
            }
          }
        }
      }
      team_sum<2 * RB>(s, p.lanes, s_sum, place);
      place ^= 1;
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const int64_t row = row0 + r * p.team_rows + row_of_team;
        const float n = rsqrtf(__fdiv_rn(s[2 * r], p.gs_f) + p.eps);
        const float muv = __fdiv_rn(s[2 * r + 1], p.gs_f) * n * n;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          if (!has[i] || row >= p.rows) continue;
          float y[E], gv[E], z[E], dy[E], dz[E];
          xc[r][i].get(y), gc[r][i].get(gv), zc[r][i].get(z);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float sg = sig[r][i][k], act = z[k] * sg;
            const float slope = sg * fmaf(z[k], 1.0f - sg, 1.0f);
            const float u = gv[k] * w[i][k];
            if constexpr (KIND == kMamba2Grad) {
              const float v = y[k] * act;
              const float dv = n * (u - v * muv);
              dy[k] = dv * act;
              dz[k] = dv * y[k] * slope;
              dw[i][k] = fmaf(gv[k], v * n, dw[i][k]);
            } else {
              const float yn = y[k] * n;
              dy[k] = n * (u * act - y[k] * muv);
              dz[k] = u * yn * slope;
              dw[i][k] = fmaf(gv[k] * act, yn, dw[i][k]);
            }
          }
          const int64_t at = c0 + (lane + i * p.lanes) * E;
          Block<T, E>::put(static_cast<T*>(p.out) + row * p.os + at, dy);
          Block<T, E>::put(static_cast<T*>(p.dgate) + row * p.dgs + at, dz);
        }
      }
    }
  }

  if constexpr (kGrad) {
    // The CTA's sums: teams on other rows of a group (ONNX: all teams) in order.
    const int teams = KIND == kOnnxGrad ? p.team_rows * p.team_groups : p.team_rows;
    const int apart = KIND == kOnnxGrad ? 1 : p.team_groups;  // teams of the same columns
    const bool first = KIND == kOnnxGrad ? team == 0 : row_of_team == 0;
    const int64_t columns = KIND == kOnnxGrad ? p.gs : p.groups * p.gs;
    const int64_t sum = KIND == kOnnxGrad ? blockIdx.y * gridDim.x + blockIdx.x : blockIdx.x;
    const int64_t col0 = KIND == kOnnxGrad ? 0 : c0;
    auto finish = [&](float (&a)[VPL][E], float* out) {
      if (teams > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
#pragma unroll
          for (int k = 0; k < E; ++k) s_acc[(i * E + k) * blockDim.x + threadIdx.x] = a[i][k];
        }
        __syncthreads();
        if (first) {
          for (int t = 1; t < teams; ++t) {
            const int from = threadIdx.x + t * apart * p.lanes;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
#pragma unroll
              for (int k = 0; k < E; ++k) a[i][k] += s_acc[(i * E + k) * blockDim.x + from];
            }
          }
        }
      }
      if (!first) return;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (!has[i]) continue;
#pragma unroll
        for (int k = 0; k < E; ++k)
          out[sum * columns + col0 + (lane + i * p.lanes) * E + k] = a[i][k];
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
  __shared__ float s_sum[2 * (kMaxThreads / 32) * 8];
  pdl_wait();
  pdl_launch_dependents();
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
template <int KIND, typename T>
int launch_kind(const Params& p, const Plan& k, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(k.slices), static_cast<unsigned>(k.blocks));
  const auto go = [&](auto kernel) {
    return mixer::launch(kernel, grid, static_cast<unsigned>(k.threads), k.smem, s, p);
  };
  if (k.vpl == 0) return go(k_norm_any<KIND, T>);
  constexpr int B = sizeof(T), V = 16 / B;
  if (k.elems == V) {
    if (k.vpl == 1) return go(k_norm<KIND, T, V, 1, rows_ahead(B, V, 1)>);
    if (k.vpl == 2) return go(k_norm<KIND, T, V, 2, rows_ahead(B, V, 2)>);
    return go(k_norm<KIND, T, V, 4, rows_ahead(B, V, 4)>);
  }
  if (k.elems == V / 2) {
    if (k.vpl == 1) return go(k_norm<KIND, T, V / 2, 1, rows_ahead(B, V / 2, 1)>);
    return go(k_norm<KIND, T, V / 2, 4, rows_ahead(B, V / 2, 4)>);
  }
  if (k.vpl == 1) return go(k_norm<KIND, T, 1, 1, rows_ahead(B, 1, 1)>);
  return go(k_norm<KIND, T, 1, 4, rows_ahead(B, 1, 4)>);
}

int launch_f32(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_f16(int kind, const Params& p, const Plan& k, cudaStream_t s);
int launch_bf16(int kind, const Params& p, const Plan& k, cudaStream_t s);

}  // namespace norms
}  // namespace ggrn
