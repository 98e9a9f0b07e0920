// ggrn_scan.cu -- the selective state space scan of the Mamba-2 mixer (one
// decay per head) for prompts and for single tokens.
//
//   dt[t] = clamp(softplus(dt_raw + dt_bias)),  e[t] = exp(dt[t] a)
//   S[t]  = e[t] S[t-1] + dt[t] x[t] (x) B[t],  y[t] = S[t] C[t] + d x[t]
//
// with S [head_dim, state_size] per head and B, C shared by the heads of a
// group.
//
// k_scan is the recurrence as it stands, for every type and size: the state
// lives in registers in f32 (4 rows of S x 16 columns per thread, a team of TL
// lanes across the columns), tokens come in blocks of 16 through shared memory
// (asynchronous copies, a block ahead), three f32x2 instructions per pair of
// state entries and token, which bound it: each takes the multiply-add pipe for
// two cycles, and the pipe is busy 59 % of the time (1025 tokens of 48 heads of
// 100 x 64 in f32: 131 us with the parts' states).
//
// A sequence longer than a part (see find_part) is cut: a first launch runs
// every part but the last of its sequence from a zero state, for its final
// state and its decay alone; k_scan_join turns those into the states at the
// parts' starts; the main launch then runs all parts at once.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "ggrn_optin.h"
#include "ggrn_scan.cuh"

namespace ggrn {
namespace scan {

// ---------------------------------------------------------------------------
// k_scan: the recurrence, token by token.
// ---------------------------------------------------------------------------
constexpr int kBlock = 16;   // tokens staged in shared memory at a time
constexpr int kCols = 16;    // state columns of a thread: 4 runs of 4, team-interleaved
constexpr int kRows = 4;     // rows of S of a thread
constexpr int kMaxThreads = 256, kMaxRows = 256;
constexpr int kMaxSmem = 96 * 1024;
constexpr int kMinPart = 64;  // rows of the shortest part worth its join

template <typename T>
__device__ __forceinline__ float ld1(const T* p) {
  return Elem<T>::load1(p, 0);
}
// Four consecutive values from shared memory, as two pairs.
struct Quad {
  F2 lo, hi;
};
__device__ __forceinline__ Quad lds4(const float* p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  return {v.x, v.y};
}
template <typename T>
__device__ __forceinline__ Quad lds4(const T* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  float a, b, c, d;
  Elem<T>::unpack2(u.x, a, b);
  Elem<T>::unpack2(u.y, c, d);
  return {pk2(a, b), pk2(c, d)};
}

// The first n of a pair, zeros behind them.
__device__ __forceinline__ F2 first_of(F2 v, int n) {
  float a, b;
  upk2(v, a, b);
  return pk2(n > 0 ? a : 0.0f, n > 1 ? b : 0.0f);
}

__device__ __forceinline__ float ld_smem(const float* p) { return *p; }
template <typename T>
__device__ __forceinline__ float ld_smem(const T* p) {
  return static_cast<float>(*p);
}

// What the host found out about the layout: bytes an asynchronous copy of a row
// of B and C, or of x, may move (16, 8, 4; 2: none, element by element).
struct Shape {
  int tl, threads, prows, ptiles;
  int bc_bytes, x_bytes;
  bool vec;        // rows of the state in 16-byte vectors
  int np;          // elements of a row of B or C in shared memory
  size_t smem;
};

// `cols` elements of a row into shared memory by one warp, BYTES at a time.
template <int BYTES, typename T>
__device__ __forceinline__ void copy_row(T* dst, const T* src, int cols) {
  const int total = cols * static_cast<int>(sizeof(T));
  const uint32_t d = smem_u32(dst);
  const char* s = reinterpret_cast<const char*>(src);
#pragma unroll 1
  for (int i = (threadIdx.x & 31) * BYTES; i < total; i += 32 * BYTES) {
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i), "l"(s + i) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d + i), "l"(s + i), "n"(BYTES)
                   : "memory");
  }
}
template <typename T>
__device__ __forceinline__ void copy_row(T* dst, const T* src, int cols, int bytes) {
  if (bytes == 16) {
    copy_row<16>(dst, src, cols);
  } else if (bytes == 8) {
    copy_row<8>(dst, src, cols);
  } else if (bytes == 4) {
    copy_row<4>(dst, src, cols);
  } else {
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < cols; i += 32) dst[i] = src[i];
  }
}

// Sums of four values over a team of TL lanes: afterwards lane l of the team
// holds the sum of value team_row<TL>(l) (TL >= 4), those of two values in v[0]
// and v[1] (TL == 2), or all four (TL == 1).
template <int TL>
__device__ __forceinline__ void team_sums(float (&v)[4], int l) {
  if constexpr (TL >= 2) {
    const bool up = l & (TL / 2);
    const float a = up ? v[0] : v[2], b = up ? v[1] : v[3];
    v[0] = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, a, TL / 2);
    v[1] = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, b, TL / 2);
  }
  if constexpr (TL >= 4) {
    const bool up = l & (TL / 4);
    const float a = up ? v[0] : v[1];
    v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, a, TL / 4);
#pragma unroll
    for (int o = TL / 8; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  }
}

// STATE_ONLY: the first launch of a cut scan.  PADS: a team's columns go on
// behind N (a form of its own: in one form for both, 1025 tokens of 48 heads of
// 100 x 64 in f32 took 134 us against 131).
template <typename T, int TL, bool STATE_ONLY, bool PADS>
__global__ void __launch_bounds__(kMaxThreads, 2) k_scan(const Params p, const Shape sh) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  pdl_wait();
  pdl_launch_dependents();
  const Part part = find_part<STATE_ONLY>(p.q, p.part, blockIdx.x);
  if (part.seq < 0) return;
  // (offsets that do not ascend may count more places than there are)
  if (part.count > 1 && part.place + (STATE_ONLY ? 1 : 0) >= p.places) return;
  const int P = p.P, N = p.N, prows = sh.prows;
  const int h = blockIdx.y, g = h / p.hpg;
  const int row0 = blockIdx.z * prows;
  const int rows_here = min(prows, P - row0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int l = tid & (TL - 1);
  const int r0 = tid / TL * kRows;           // this thread's first row of the tile
  // shared memory: two blocks of B, C and x rows as they come; one of (dt x)
  // as pairs of equal halves, in whose places the y are left; one of B and C in
  // f32 if T is not; dt and decays
  constexpr bool kWiden = sizeof(T) == 2;
  T* sB = reinterpret_cast<T*>(smem_raw);    // [2][kBlock][np]
  T* sC = sB + 2 * kBlock * sh.np;
  T* sX = sC + 2 * kBlock * sh.np;           // [2][kBlock][prows]
  float* sXX = reinterpret_cast<float*>(sX + 2 * kBlock * prows);  // [kBlock][prows][2]
  float* sBf = sXX + 2 * kBlock * prows;     // [kBlock][np]
  float* sCf = sBf + kBlock * sh.np;
  float* sDt = kWiden ? sCf + kBlock * sh.np : sBf;  // [2][kBlock] dt, decay
  const float a = __ldg(p.a + h), dbias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.0f;
  const float dskip = p.d ? __ldg(p.d + h) : 0.0f;
  const int64_t slot = seq_slot(p.q, part.seq);
  const int64_t PN = static_cast<int64_t>(P) * N;

  const T* x = static_cast<const T*>(p.x) + static_cast<int64_t>(h) * P + row0;
  const T* b = static_cast<const T*>(p.b) + static_cast<int64_t>(g) * N;
  const T* c = static_cast<const T*>(p.c) + static_cast<int64_t>(g) * N;
  const T* dtp = static_cast<const T*>(p.dt) + h;
  T* out = static_cast<T*>(p.out) + static_cast<int64_t>(h) * P + row0;

  auto fetch = [&](int64_t t0, int buf) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(kBlock), part.end - t0));
    const T* bt = b + (t0 + warp) * p.bs;
    const T* ct = c + (t0 + warp) * p.cs;
    const T* xt = x + (t0 + warp) * p.xs;
    int row = buf * kBlock + warp;
#pragma unroll 1
    for (int t = warp; t < nt; t += warps, row += warps) {
      if (sh.bc_bytes == 16 && sh.x_bytes == 16) {  // as a rule
        copy_row<16>(sB + row * sh.np, bt, N);
        if (!STATE_ONLY) copy_row<16>(sC + row * sh.np, ct, N);
        copy_row<16>(sX + row * prows, xt, rows_here);
      } else {
        copy_row(sB + row * sh.np, bt, N, sh.bc_bytes);
        if (!STATE_ONLY) copy_row(sC + row * sh.np, ct, N, sh.bc_bytes);
        copy_row(sX + row * prows, xt, rows_here, sh.x_bytes);
      }
      bt += warps * p.bs, ct += warps * p.cs, xt += warps * p.xs;
    }
  };
  // columns behind N and rows behind the tile's are zeros throughout
#pragma unroll 1
  for (int t = warp; t < 2 * kBlock; t += warps) {
#pragma unroll 1
    for (int i = N + lane; i < sh.np; i += 32)
      Elem<T>::store1(sB + t * sh.np, i, 0.0f), Elem<T>::store1(sC + t * sh.np, i, 0.0f);
#pragma unroll 1
    for (int i = rows_here + lane; i < prows; i += 32) Elem<T>::store1(sX + t * prows, i, 0.0f);
  }
  float raw = 0.0f;
  if (part.begin < part.end) {
    fetch(part.begin, 0);
    if (part.begin + tid < part.end && tid < kBlock) raw = ld1(dtp + (part.begin + tid) * p.dts);
  }

  F2 s[kRows][kCols / 2];  // columns 4 (TL k + l) .. in two pairs
  // the state this part starts from: the workspace's for a cut sequence,
  // else the pool's or zeros
  const float* from = nullptr;
  if (!STATE_ONLY) {
    if (part.count > 1) from = p.ws + (part.place * p.H + h) * PN;
    else if (slot >= 0 && seq_resumes(p.q, part.seq)) from = p.state + slot * p.slot_stride + h * PN;
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float* at = from + static_cast<int64_t>(row0 + r0 + r) * N + l * 4;
    const bool here = from && r0 + r < rows_here;
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j) {
      float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int left = here ? N - (j * TL + l) * 4 : 0;
      if (sh.vec) {
        if (left > 0) {
          const float4 v = *reinterpret_cast<const float4*>(at + j * TL * 4);
          q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) q[i] = at[j * TL * 4 + i];
      }
      s[r][2 * j] = pk2(q[0], q[1]), s[r][2 * j + 1] = pk2(q[2], q[3]);
    }
  }
  float log_decay = 0.0f;  // STATE_ONLY, threads of the first block of tokens

  // K tokens from token t of the block on.  HOLD keeps the columns behind N
  // zeros where 0 times a value that is not finite would leave a NaN, which
  // their zeros in C would carry into y.
  using Staged = typename std::conditional<kWiden, float, T>::type;
  auto tokens = [&](auto k_tokens, auto hold, int t, const Staged* bt, const Staged* ct,
                    const float* dts) __attribute__((always_inline)) {
    constexpr int K = decltype(k_tokens)::value;
    constexpr bool HOLD = decltype(hold)::value;
    bt += t * sh.np + l * 4;
    ct += t * sh.np + l * 4;
    float* xt = sXX + (t * prows + r0) * 2;
    F2 ee[K], xx[K][kRows], yy[K][kRows];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ee[k] = *reinterpret_cast<const F2*>(dts + kBlock + 2 * (t + k));
      const Quad lo = lds4(xt + k * prows * 2), hi = lds4(xt + k * prows * 2 + 4);
      xx[k][0] = lo.lo, xx[k][1] = lo.hi, xx[k][2] = hi.lo, xx[k][3] = hi.hi;
    }
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Quad bv = lds4(bt + k * sh.np + j * TL * 4);
        Quad cv = {0, 0};
        if (!STATE_ONLY) cv = lds4(ct + k * sh.np + j * TL * 4);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          s[r][2 * j] = fma2(s[r][2 * j], ee[k], mul2(bv.lo, xx[k][r]));
          s[r][2 * j + 1] = fma2(s[r][2 * j + 1], ee[k], mul2(bv.hi, xx[k][r]));
          if constexpr (HOLD) {
            const int left = N - (j * TL + l) * 4;
            s[r][2 * j] = first_of(s[r][2 * j], left);
            s[r][2 * j + 1] = first_of(s[r][2 * j + 1], left - 2);
          }
          if (!STATE_ONLY) {
            yy[k][r] = j == 0 ? mul2(s[r][0], cv.lo) : fma2(s[r][2 * j], cv.lo, yy[k][r]);
            yy[k][r] = fma2(s[r][2 * j + 1], cv.hi, yy[k][r]);
          }
        }
      }
    if constexpr (!STATE_ONLY) {
      float y[K][kRows];
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float y0, y1;
          upk2(yy[k][r], y0, y1);
          y[k][r] = y0 + y1;
        }
        team_sums<TL>(y[k], l);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        // (only this team reads these places)
        float* yt = xt + k * prows * 2;
        if constexpr (TL >= 4) {
          // the lane whose low bits are zero writes the row of its high bits
          if ((l & (TL / 4 - 1)) == 0)
            yt[(l & (TL / 2) ? 4 : 0) + (l & (TL / 4) ? 2 : 0)] = y[k][0];
        } else if constexpr (TL == 2) {
          yt[4 * l] = y[k][0], yt[4 * l + 2] = y[k][1];
        } else {
#pragma unroll
          for (int r = 0; r < kRows; ++r) yt[2 * r] = y[k][r];
        }
      }
    }
  };

  int buf = 0;
#pragma unroll 1
  for (int64_t t0 = part.begin; t0 < part.end; t0 += kBlock, buf ^= 1) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(kBlock), part.end - t0));
    float* dts = sDt + buf * 3 * kBlock;  // dt; decays, twice each
    F2 odd = 0;  // NaN where a decay or a dt x of the block is not finite
    if (tid < nt) {
      const float dt = dt_of(raw, dbias, p), e = expf(dt * a);
      if constexpr (PADS) odd = pk2(e * 0.0f, 0.0f);
      dts[tid] = dt;
      *reinterpret_cast<float2*>(dts + kBlock + 2 * tid) = make_float2(e, e);
      if (STATE_ONLY) log_decay = fmaf(dt, a, log_decay);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (t0 + kBlock < part.end) {
      fetch(t0 + kBlock, buf ^ 1);
      if (t0 + kBlock + tid < part.end && tid < kBlock)
        raw = ld1(dtp + (t0 + kBlock + tid) * p.dts);
    }
    const T* bb = sB + buf * kBlock * sh.np;
    const T* cb = sC + buf * kBlock * sh.np;
    const T* xb = sX + buf * kBlock * prows;
#pragma unroll 1
    for (int t = warp; t < nt; t += warps) {
      const F2 dd = pk2(dts[t], dts[t]);
#pragma unroll 1
      for (int i = lane * 4; i < prows; i += 128) {
        const Quad q = lds4(xb + t * prows + i);
        const F2 lo = mul2(q.lo, dd), hi = mul2(q.hi, dd);
        if constexpr (PADS) odd = fma2(lo, 0, fma2(hi, 0, odd));
        float v[4];
        upk2(lo, v[0], v[1]);
        upk2(hi, v[2], v[3]);
        float4* to = reinterpret_cast<float4*>(sXX + (t * prows + i) * 2);
        to[0] = make_float4(v[0], v[0], v[1], v[1]);
        to[1] = make_float4(v[2], v[2], v[3], v[3]);
      }
      if constexpr (kWiden) {
#pragma unroll 1
        for (int i = lane * 4; i < sh.np; i += 128) {
          const int at = t * sh.np + i;
          const Quad q = lds4(bb + at);
          *reinterpret_cast<ulonglong2*>(sBf + at) = make_ulonglong2(q.lo, q.hi);
          if (!STATE_ONLY) {
            const Quad r = lds4(cb + at);
            *reinterpret_cast<ulonglong2*>(sCf + at) = make_ulonglong2(r.lo, r.hi);
          }
        }
      }
    }
    bool hold = false;
    if constexpr (PADS) {
      float odd0, odd1;
      upk2(odd, odd0, odd1);
      hold = __syncthreads_or(odd0 != odd0 || odd1 != odd1) != 0;
    } else {
      __syncthreads();
    }
    // tokens by pairs, for more instructions that do not wait for one another
    const Staged* bt;
    const Staged* ct;
    if constexpr (kWiden) {
      bt = sBf, ct = sCf;
    } else {
      bt = bb, ct = cb;
    }
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    int t = 0;
    if constexpr (PADS)
      if (hold)
#pragma unroll 1
        for (; t < nt; ++t) tokens(One(), std::true_type(), t, bt, ct, dts);
#pragma unroll 1
    for (; t + 2 <= nt; t += 2) tokens(Two(), std::false_type(), t, bt, ct, dts);
    if (t < nt) tokens(One(), std::false_type(), t, bt, ct, dts);
    __syncthreads();
    if (!STATE_ONLY) {
      T* ot = out + (t0 + warp) * p.os;
#pragma unroll 1
      for (int t = warp; t < nt; t += warps, ot += warps * p.os)
#pragma unroll 1
        for (int r = lane; r < rows_here; r += 32)
          Elem<T>::store1(ot, r, fmaf(dskip, ld_smem(xb + t * prows + r), sXX[(t * prows + r) * 2]));
    }
  }

  // where the state goes: the next part's place in the workspace, or the pool
  float* to = nullptr;
  if (STATE_ONLY) {
    to = p.ws + ((part.place + 1) * p.H + h) * PN;
    if (warp == 0 && blockIdx.z == 0) {
#pragma unroll
      for (int o = kBlock / 2; o > 0; o >>= 1)
        log_decay += __shfl_xor_sync(0xffffffffu, log_decay, o);
      if (lane == 0) p.ws_decay[part.place * p.H + h] = expf(log_decay);
    }
  } else if (part.index == part.count - 1 && slot >= 0) {
    to = p.state + slot * p.slot_stride + h * PN;
  }
  if (!to) return;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float* at = to + static_cast<int64_t>(row0 + r0 + r) * N + l * 4;
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j) {
      float q[4];
      upk2(s[r][2 * j], q[0], q[1]);
      upk2(s[r][2 * j + 1], q[2], q[3]);
      const int left = r0 + r < rows_here ? N - (j * TL + l) * 4 : 0;
      if (sh.vec) {
        if (left > 0)
          *reinterpret_cast<float4*>(at + j * TL * 4) = make_float4(q[0], q[1], q[2], q[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) at[j * TL * 4 + i] = q[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// k_scan_join: the states at the starts of a cut sequence's parts.  The place
// of part i > 0 holds what part i - 1 adds to the state from a zero start; a
// thread takes four entries of a state (V = 4: 16 bytes) or one through the
// parts of its sequence (1025 rows in parts of 64, 48 heads of 100 x 64: 10 us,
// the latency of its loads).  grid: (blocks of entries, heads, cut sequences:
// there are at most rows / part).
// ---------------------------------------------------------------------------
// Parts whose entries are in flight (eight cost registers, and with them warps:
// 5 % of a ragged scan's time).
constexpr int kJoinAhead = 2;

template <int V>
__global__ void __launch_bounds__(256) k_scan_join(const Params p) {
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.y;
  // the blockIdx.z-th sequence of more than one part, and its first place
  int64_t seq = -1, first = 0, count = 0;
  if (!p.q.cu) {
    seq = blockIdx.z;
    count = parts_of(p.q.each, p.part);
    first = seq * count;
  } else {
    const int lane = threadIdx.x & 31;
    int before = 0;  // cut sequences
    for (int64_t base = 0; base < p.q.seqs && seq < 0; base += 32) {
      int64_t b = 0, e = 0;
      if (base + lane < p.q.seqs) seq_range(p.q, base + lane, b, e);
      const int mine = static_cast<int>(part_counts(e - b, p.part) >> 32);  // 0: not cut
      const unsigned cut = __ballot_sync(0xffffffffu, mine > 0);
      const int found = __popc(cut);
      const unsigned here =
          __ballot_sync(0xffffffffu, mine > 0 && before + __popc(cut & ((2u << lane) - 1)) ==
                                                     static_cast<int>(blockIdx.z) + 1);
      const int l = here ? __ffs(here) - 1 : 32;
      int sum = lane < l ? mine : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      first += sum;
      if (here) {
        seq = base + l;
        count = __shfl_sync(0xffffffffu, mine, l);
      }
      before += found;
    }
  }
  if (seq < 0) return;
  if (first + count > p.places) return;  // offsets that do not ascend: no places for these
  const int64_t PN = static_cast<int64_t>(p.P) * p.N;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * V;
  if (i >= PN) return;
  const int64_t slot = seq_slot(p.q, seq);
  using W = typename std::conditional<V == 4, float4, float>::type;
  W s{};
  if (slot >= 0 && seq_resumes(p.q, seq)) {
    const float* from = p.state + slot * p.slot_stride + static_cast<int64_t>(h) * PN + i;
    if constexpr (V == 4) {  // (the pool need not be aligned)
      s = make_float4(from[0], from[1], from[2], from[3]);
    } else {
      s = *from;
    }
  }
  float* w = p.ws + (first * p.H + h) * PN + i;
  const float* decay = p.ws_decay + first * p.H + h;
  *reinterpret_cast<W*>(w) = s;
  const int64_t stride = static_cast<int64_t>(p.H) * PN;
  for (int64_t k = 0; k + 1 < count; k += kJoinAhead) {
    W add[kJoinAhead];
    float d[kJoinAhead];
    const int n = static_cast<int>(min(count - 1 - k, static_cast<int64_t>(kJoinAhead)));
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j)
      if (j < n) {
        d[j] = decay[(k + j) * p.H];
        add[j] = *reinterpret_cast<const W*>(w + (j + 1) * stride);
      }
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j)
      if (j < n) {
        if constexpr (V == 4) {
          s.x = fmaf(s.x, d[j], add[j].x), s.y = fmaf(s.y, d[j], add[j].y);
          s.z = fmaf(s.z, d[j], add[j].z), s.w = fmaf(s.w, d[j], add[j].w);
        } else {
          s = fmaf(s, d[j], add[j]);
        }
        *reinterpret_cast<W*>(w + (j + 1) * stride) = s;
      }
    w += kJoinAhead * stride;
  }
}

// ---------------------------------------------------------------------------
// k_scan_step: one token.  Bound by the state's bytes (8 per entry, read and
// written once).  A warp takes kStepRows rows of one head's S at a time, all
// their loads in flight before the first is used; the lanes hold B and C of
// their columns.  128 sequences of 96 heads of 80 x 128: 154 us, 97 % of the
// rate of a plain copy; one sequence: 3.8 us, of which 1.2 are its bytes.  VEC:
// lanes take 4 columns (16 bytes), state_size a multiple of 4 and the pool
// 16-byte aligned; else one column each.
// ---------------------------------------------------------------------------
constexpr int kStepRows = 4;
constexpr int kStepThreads = 128;

template <typename T, int CH, bool VEC>
__global__ void __launch_bounds__(kStepThreads) k_scan_step(const Params p, const int tl,
                                                            const int tile) {
  constexpr int E = VEC ? 4 : 1;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = blockIdx.x;
  const int h = blockIdx.y, g = h / p.hpg, P = p.P, N = p.N;
  const int64_t slot = seq_slot(p.q, i);
  if (slot < 0) return;
  const int l = threadIdx.x & (tl - 1);          // lane of the team of a row
  const int team = threadIdx.x / tl, teams = kStepThreads / tl;
  const int p0 = blockIdx.z * tile;
  const int p1 = min(P, p0 + tile);
  const T* x = static_cast<const T*>(p.x) + i * p.xs + static_cast<int64_t>(h) * P;
  T* out = static_cast<T*>(p.out) + i * p.os + static_cast<int64_t>(h) * P;
  float* st = p.state + slot * p.slot_stride + static_cast<int64_t>(h) * P * N;

  // the first rows' states are in flight before anything else is waited for
  float s[kStepRows][CH * E];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
      const int row = r0 + r * teams;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int n = (k * tl + l) * E;
        if (row < p1 && n < N) {
          if constexpr (VEC) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(st + static_cast<int64_t>(row) * N + n));
            s[r][k * 4] = v.x, s[r][k * 4 + 1] = v.y, s[r][k * 4 + 2] = v.z, s[r][k * 4 + 3] = v.w;
          } else {
            s[r][k] = st[static_cast<int64_t>(row) * N + n];
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) s[r][k * E + e] = 0.0f;
        }
      }
    }
  };
  fetch(p0 + team);
  float bv[CH * E], cv[CH * E];
  const T* b = static_cast<const T*>(p.b) + i * p.bs + static_cast<int64_t>(g) * N;
  const T* c = static_cast<const T*>(p.c) + i * p.cs + static_cast<int64_t>(g) * N;
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int n = (k * tl + l) * E + e;
      bv[k * E + e] = n < N ? ld1(b + n) : 0.0f;
      cv[k * E + e] = n < N ? ld1(c + n) : 0.0f;
    }
  const float dt = dt_of(ld1(static_cast<const T*>(p.dt) + i * p.dts + h),
                         p.dt_bias ? __ldg(p.dt_bias + h) : 0.0f, p);
  const float e = expf(dt * __ldg(p.a + h));
  const float dskip = p.d ? __ldg(p.d + h) : 0.0f;
  // every team of a warp makes the same number of rounds (the shuffles)
  for (int r0 = p0; r0 < p1; r0 += kStepRows * teams) {
    if (r0 > p0) fetch(r0 + team);
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
      const int row = r0 + team + r * teams;
      const float xv = row < p1 ? ld1(x + row) : 0.0f;
      const float xd = dt * xv;
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < CH * E; ++k) {
        // (columns behind N stay zeros whatever dt x and the decay are)
        s[r][k] = (k / E * tl + l) * E < N ? fmaf(s[r][k], e, xd * bv[k]) : 0.0f;
        y = fmaf(s[r][k], cv[k], y);
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int n = (k * tl + l) * E;
        if (row < p1 && n < N) {
          if constexpr (VEC)
            __stcs(reinterpret_cast<float4*>(st + static_cast<int64_t>(row) * N + n),
                   make_float4(s[r][k * 4], s[r][k * 4 + 1], s[r][k * 4 + 2], s[r][k * 4 + 3]));
          else
            st[static_cast<int64_t>(row) * N + n] = s[r][k];
        }
      }
      for (int o = tl >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (l == 0 && row < p1) Elem<T>::store1(out + row, 0, fmaf(dskip, xv, y));
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int pow2_at_least(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// k_scan's CTAs.
Shape shape_of(int P, int N, int es) {
  Shape s = {};
  s.tl = pow2_at_least((N + kCols - 1) / kCols);
  const int most = std::min(kMaxThreads / s.tl * kRows, kMaxRows);  // rows of the largest CTA
  s.ptiles = (P + most - 1) / most;
  const int teams = ((P + s.ptiles - 1) / s.ptiles + kRows - 1) / kRows;
  s.threads = (teams * s.tl + 31) / 32 * 32;
  s.prows = s.threads / s.tl * kRows;
  s.ptiles = (P + s.prows - 1) / s.prows;
  s.np = s.tl * kCols;
  s.smem = static_cast<size_t>(es) * 2 * kBlock * (2 * s.np + s.prows) +
           4 * static_cast<size_t>(kBlock) * (2 * s.prows + (es == 2 ? 2 * s.np : 0) + 6);
  return s;
}
// The widest copy that every row of these layouts allows.
int copy_bytes(std::initializer_list<int64_t> at) {
  int64_t all = 16;
  for (int64_t v : at) all |= v;
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

// Rows of a part of k_scan: long sequences are cut until the launch holds
// about six CTAs for each SM.  4096 tokens of 96 heads of 80 x 128 in f16:
// 1365 us with four, 1283 with six, 1254 with eight, whose states take a third
// more workspace; 1025 of 48 heads of 100 x 64 in f32: 132.5, 131.5, 132.
int64_t part_rows(int64_t rows, int64_t ctas_per_part) {
  const int64_t want = 6 * static_cast<int64_t>(device_sms());
  const int64_t parts = std::max<int64_t>(1, want / std::max<int64_t>(1, ctas_per_part));
  const int64_t part = (rows + parts - 1) / parts;
  return std::max<int64_t>(kMinPart, (part + kBlock - 1) / kBlock * kBlock);
}

// Sequences of more than one part that a call can have (a grid's third
// dimension); parts of calls with more sequences are long enough for it.
constexpr int64_t kMaxCut = 65535;

// The most rows a sequence can have.
int64_t longest(const ggrn_scan_call& c) {
  return c.cu_seqlens || c.seqs <= 0 ? c.rows : c.rows / c.seqs;
}

struct Layout {
  bool tc;                  // on the tensor cores
  int64_t part, parts;      // rows of a part; the most parts there can be
  int64_t places;           // the most of them that are of cut sequences
  bool cut;                 // whether a sequence may have more than one
  int64_t state_bytes, bytes;
};
Layout layout_of(const ggrn_scan_call& c) {
  Layout l;
  const Shape s = shape_of(static_cast<int>(c.head_dim), static_cast<int>(c.state_size),
                           mixer::elem_bytes(c.dtype));
  l.tc = tc_covers(c);
  l.part = l.tc ? tc_part_rows(c, longest(c)) : part_rows(c.rows, c.heads * s.ptiles);
  if (longest(c) > INT32_MAX) l.part = longest(c);  // (the kernels count parts in 32 bits)
  // the join's grid holds kMaxCut sequences of more than one part
  if (c.seqs > kMaxCut) {
    if (!c.cu_seqlens) l.part = std::max(l.part, longest(c));
    else if (c.rows / l.part > kMaxCut) l.part = (c.rows / kMaxCut / 128 + 1) * 128;
  }
  l.cut = longest(c) > l.part;
  if (!l.cut) l.part = std::max<int64_t>(1, longest(c));
  // (a sequence of n > 0 rows has (n - 1) / part + 1, an empty one has one)
  l.parts = (c.rows > 0 ? (c.rows - 1) / l.part : 0) + c.seqs;
  if (!c.cu_seqlens && c.seqs > 0)
    l.parts = c.seqs * std::max<int64_t>(1, (c.rows / c.seqs + l.part - 1) / l.part);
  l.places = l.state_bytes = l.bytes = 0;
  if (l.cut) {
    l.places = c.cu_seqlens ? std::min(l.parts, 2 * (c.rows / l.part)) : l.parts;
    const __int128 bytes = static_cast<__int128>(l.places) * c.heads * c.head_dim * c.state_size * 4;
    if (bytes > INT64_MAX / 2) {  // (more than there can be)
      l.bytes = INT64_MAX;
      return l;
    }
    l.state_bytes = (static_cast<int64_t>(bytes) + 15) / 16 * 16;
    l.bytes = l.state_bytes + (l.places * c.heads * 4 + 15) / 16 * 16;
  }
  return l;
}

// Sizes alone (what ggrn_scan_workspace_bytes looks at).
int check_sizes(const ggrn_scan_call& c) {
  if (c.dtype != kF32 && c.dtype != kF16 && c.dtype != kBF16) return GGRN_ERR_DTYPE;
  if (c.rows < 0 || c.heads <= 0 || c.head_dim <= 0 || c.groups <= 0 || c.state_size <= 0 ||
      c.heads % c.groups != 0)
    return GGRN_ERR_SHAPE;
  if (c.state_size > 256 || c.heads > 65535 || c.head_dim > 65535) return GGRN_ERR_UNSUPPORTED;
  return GGRN_OK;
}

int check(const ggrn_scan_call& c, bool step, Params* p) {
  int st = check_sizes(c);
  if (st != GGRN_OK) return st;
  if (!(c.dt_min >= 0.0f) || !(c.dt_max >= c.dt_min)) return GGRN_ERR_ARG;
  const int es = mixer::elem_bytes(c.dtype);
  const int64_t width = c.heads * c.head_dim, gn = c.groups * c.state_size;
  const int64_t held = width * c.state_size;
  st = mixer::check_seqs(c.rows, c.seqs, c.cu_seqlens, c.state, c.slots, c.resume, c.state_slots,
                         held, c.state_slot_stride, step, &p->q);
  if (st != GGRN_OK) return st;
  mixer::Buffer x, dt, b, cc, out, state;
  if (!mixer::extent(c.x, c.rows, width, c.x_row_stride, es, &x) ||
      !mixer::extent(c.dt, c.rows, c.heads, c.dt_row_stride, es, &dt) ||
      !mixer::extent(c.b, c.rows, gn, c.b_row_stride, es, &b) ||
      !mixer::extent(c.c, c.rows, gn, c.c_row_stride, es, &cc) ||
      !mixer::extent(c.out, c.rows, width, c.out_row_stride, es, &out) ||
      !mixer::extent(c.state, c.state ? c.state_slots : 0, held, c.state_slot_stride, 4, &state))
    return GGRN_ERR_SHAPE;
  if (c.rows == 0 && (!c.state || p->q.seqs == 0)) return GGRN_OK;
  if (!c.a || (c.rows > 0 && (!c.x || !c.dt || !c.b || !c.c || !c.out))) return GGRN_ERR_NULL;
  for (const void* q : {c.x, c.dt, c.b, c.c, static_cast<const void*>(c.out)})
    if (!mixer::aligned_to(q, es)) return GGRN_ERR_ALIGN;
  for (const float* q : {c.a, c.d, c.dt_bias, static_cast<const float*>(c.state)})
    if (!mixer::aligned_to(q, 4)) return GGRN_ERR_ALIGN;
  const int64_t n = p->q.seqs;
  const mixer::Buffer ins[] = {x,
                               dt,
                               b,
                               cc,
                               {c.a, c.heads * 4},
                               {c.d, c.heads * 4},
                               {c.dt_bias, c.heads * 4},
                               {p->q.cu, (n + 1) * 4},
                               {p->q.slots, n * 4},
                               {p->q.resume, n}};
  const mixer::Buffer ws = {step ? nullptr : c.workspace, c.workspace_bytes};
  for (const mixer::Buffer& o : {out, state, ws})
    for (const mixer::Buffer& i : ins)
      if (mixer::overlap(o, i)) return GGRN_ERR_OVERLAP;
  if (mixer::overlap(out, state) || mixer::overlap(out, ws) || mixer::overlap(state, ws))
    return GGRN_ERR_OVERLAP;
  p->x = c.x, p->dt = c.dt, p->b = c.b, p->c = c.c;
  p->a = c.a, p->d = c.d, p->dt_bias = c.dt_bias;
  p->out = c.out;
  p->state = c.state;
  const bool many = c.rows > 1;
  p->xs = many ? c.x_row_stride : 0, p->dts = many ? c.dt_row_stride : 0;
  p->bs = many ? c.b_row_stride : 0, p->cs = many ? c.c_row_stride : 0;
  p->os = many ? c.out_row_stride : 0;
  p->slot_stride = c.state_slots > 1 ? c.state_slot_stride : 0;
  p->H = static_cast<int>(c.heads), p->P = static_cast<int>(c.head_dim);
  p->N = static_cast<int>(c.state_size);
  p->hpg = static_cast<int>(c.heads / c.groups);
  p->dt_min = c.dt_min, p->dt_max = c.dt_max;
  p->softplus = c.dt_softplus;
  return GGRN_OK;
}

template <typename T, int TL>
int run_team(const Params& p, const Shape& sh, const Layout& l, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(l.parts), static_cast<unsigned>(p.H),
                  static_cast<unsigned>(sh.ptiles));
  if (sh.smem > 48 * 1024) {  // wide states in f32: up to 84 KB
    cudaError_t e = allow_shared_memory<k_scan<T, TL, true, false>>(kMaxSmem);
    if (e == cudaSuccess) e = allow_shared_memory<k_scan<T, TL, false, false>>(kMaxSmem);
    if (e == cudaSuccess) e = allow_shared_memory<k_scan<T, TL, false, true>>(kMaxSmem);
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return GGRN_ERR_CUDA;
    }
  }
  if (l.cut) {
    int st = mixer::launch(k_scan<T, TL, true, false>, dim3(inner_parts(p), grid.y, grid.z),
                           sh.threads, sh.smem, s, p, sh);
    if (st != GGRN_OK) return st;
    st = launch_join(p, s);
    if (st != GGRN_OK) return st;
  }
  // (the states' columns behind N are not stored: the first launch needs no PADS)
  return mixer::launch(p.N < sh.np ? k_scan<T, TL, false, true> : k_scan<T, TL, false, false>, grid,
                       sh.threads, sh.smem, s, p, sh);
}

template <typename T>
int run_typed(const Params& p, const Layout& l, cudaStream_t s) {
  constexpr int64_t es = sizeof(T);
  Shape sh = shape_of(p.P, p.N, es);
  if (l.parts > INT32_MAX || sh.ptiles > 65535) return GGRN_ERR_UNSUPPORTED;
  auto at = [](const void* q) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(q)); };
  sh.bc_bytes = copy_bytes({at(p.b), at(p.c), p.bs * es, p.cs * es, p.N * es});
  // (a head's columns start at multiples of P, a tile's of prows)
  sh.x_bytes = copy_bytes({at(p.x), p.xs * es, p.P * es, sh.prows * es});
  sh.vec = p.N % 4 == 0 && (!p.state || (mixer::aligned_to(p.state, 16) && p.slot_stride % 4 == 0));
  switch (sh.tl) {
    case 1: return run_team<T, 1>(p, sh, l, s);
    case 2: return run_team<T, 2>(p, sh, l, s);
    case 4: return run_team<T, 4>(p, sh, l, s);
    case 8: return run_team<T, 8>(p, sh, l, s);
    default: return run_team<T, 16>(p, sh, l, s);
  }
}

template <typename T>
int step_typed(const Params& p, cudaStream_t s) {
  const bool vec = p.N % 4 == 0 && mixer::aligned_to(p.state, 16) && p.slot_stride % 4 == 0;
  const int lanes = (p.N + (vec ? 3 : 0)) / (vec ? 4 : 1);
  const int tl = std::min(32, pow2_at_least(lanes));
  const int ch = (lanes + tl - 1) / tl;  // 1, 2 (vectors) or 1..8 (single columns)
  // one round of rows per CTA while the launch is small, else two
  const int round = kStepRows * (kStepThreads / tl);
  const int64_t rounds = p.q.rows * p.H * ((p.P + round - 1) / round);
  const int tile = rounds > 16 * device_sms() ? 2 * round : round;
  const int64_t tiles = (p.P + tile - 1) / tile;
  if (p.q.rows > INT32_MAX || tiles > 65535) return GGRN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(p.q.rows), static_cast<unsigned>(p.H),
                  static_cast<unsigned>(tiles));
  if (vec)
    return ch == 1 ? mixer::launch(k_scan_step<T, 1, true>, grid, kStepThreads, 0, s, p, tl, tile)
                   : mixer::launch(k_scan_step<T, 2, true>, grid, kStepThreads, 0, s, p, tl, tile);
  if (ch <= 2) return mixer::launch(k_scan_step<T, 2, false>, grid, kStepThreads, 0, s, p, tl, tile);
  return mixer::launch(k_scan_step<T, 8, false>, grid, kStepThreads, 0, s, p, tl, tile);
}

int run(const ggrn_scan_call* call, bool step, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_scan_call& c = *call;
  Params p = {};
  const int st = check(c, step, &p);
  if (st != GGRN_OK || (c.rows == 0 && (!c.state || p.q.seqs == 0))) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step) {
    if (c.dtype == kF32) return step_typed<float>(p, s);
    if (c.dtype == kF16) return step_typed<__half>(p, s);
    return step_typed<__nv_bfloat16>(p, s);
  }
  const Layout l = layout_of(c);
  if (l.bytes > 0) {
    if (!c.workspace) return GGRN_ERR_NULL;
    if (!mixer::aligned_to(c.workspace, 16)) return GGRN_ERR_ALIGN;
    if (c.workspace_bytes < l.bytes) return GGRN_ERR_ARG;
    p.ws = static_cast<float*>(c.workspace);
    p.ws_decay = p.ws + l.state_bytes / 4;
  }
  p.part = l.part;
  p.parts = l.parts;
  p.places = l.places;
  if (l.tc) {
    if (l.parts > INT32_MAX) return GGRN_ERR_UNSUPPORTED;
    return tc_run(c, p, l.cut, s);
  }
  if (c.dtype == kF32) return run_typed<float>(p, l, s);
  if (c.dtype == kF16) return run_typed<__half>(p, l, s);
  return run_typed<__nv_bfloat16>(p, l, s);
}

int launch_join(const Params& p, cudaStream_t s) {
  const int64_t pn = static_cast<int64_t>(p.P) * p.N;
  const int v = pn % 4 == 0 ? 4 : 1;
  const int64_t cut = std::min(p.q.seqs, p.q.cu ? p.q.rows / p.part : p.q.seqs);
  const dim3 grid(static_cast<unsigned>((pn / v + 255) / 256), static_cast<unsigned>(p.H),
                  static_cast<unsigned>(cut));
  return v == 4 ? mixer::launch(k_scan_join<4>, grid, 256, 0, s, p)
                : mixer::launch(k_scan_join<1>, grid, 256, 0, s, p);
}

}  // namespace scan

int check_scan(const ggrn_scan_call& c, bool step) {
  scan::Params p = {};
  return scan::check(c, step, &p);
}

}  // namespace ggrn

extern "C" int ggrn_scan(const ggrn_scan_call* call, void* cuda_stream) {
  return ggrn::scan::run(call, false, cuda_stream);
}
extern "C" int ggrn_scan_step(const ggrn_scan_call* call, void* cuda_stream) {
  return ggrn::scan::run(call, true, cuda_stream);
}
// One launch of the tensor-core kernel whose B and C never come.  Without a pool
// and cuts, so that nothing is written.
extern "C" int ggrn_selftest_scan_timeout(const ggrn_scan_call* call, void* cuda_stream) {
  using namespace ggrn;
  using namespace ggrn::scan;
  if (!call) return GGRN_ERR_ARG;
  const ggrn_scan_call& c = *call;
  Params p = {};
  const int st = check(c, false, &p);
  if (st != GGRN_OK) return st;
  if (c.rows == 0) return GGRN_ERR_SHAPE;
  const Layout l = layout_of(c);
  if (!l.tc || l.cut || c.state) return GGRN_ERR_UNSUPPORTED;
  p.part = l.part;
  p.parts = l.parts;
  return tc_run(c, p, false, static_cast<cudaStream_t>(cuda_stream), /*no_copies=*/true);
}
extern "C" int64_t ggrn_scan_workspace_bytes(const ggrn_scan_call* call) {
  if (!call || ggrn::scan::check_sizes(*call) != GGRN_OK ||
      !ggrn::mixer::counts_ok(call->rows, call->seqs, call->cu_seqlens != nullptr))
    return 0;
  return ggrn::scan::layout_of(*call).bytes;
}
