// ggrn_scan.cuh -- parameters and helpers shared by the scan's kernels.
#pragma once

#include "ggrn_mixer.cuh"

namespace ggrn {
namespace scan {

struct Params {
  const void* x;
  const void* dt;
  const void* b;
  const void* c;
  const float* a;
  const float* d;
  const float* dt_bias;
  void* out;
  float* state;
  float* ws;        // by place: states at the starts of parts, [places][H][P][N]
  float* ws_decay;  // decays over parts, [places][H]
  Seqs q;
  int64_t xs, dts, bs, cs, os, slot_stride;
  int64_t part, parts, places;
  int H, P, N, hpg;  // hpg: heads per group
  float dt_min, dt_max;
  int softplus;
};

// f32 pairs kept in one 64-bit register: the arithmetic on values that are
// pairs from their load on needs no moves.
using F2 = unsigned long long;
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// dt of one token and head: softplus as log1p(exp(v)), v itself from 20 on
// (the difference is below 2^-28 of it); a NaN stays one.
__device__ __forceinline__ float dt_of(float raw, float bias, const Params& p) {
  float v = raw + bias;
  if (p.softplus) v = v > 20.0f ? v : log1pf(expf(v));
  v = v < p.dt_min ? p.dt_min : v;
  return v > p.dt_max ? p.dt_max : v;
}

// The most parts there can be that are not the last of their sequence.
inline unsigned inner_parts(const Params& p) {
  return static_cast<unsigned>(p.q.cu ? p.q.rows / p.part : p.parts - p.q.seqs);
}

// Enqueue k_scan_join (the states at the parts' starts).
int launch_join(const Params& p, cudaStream_t s);

// The tensor-core kernels (ggrn_scan_tc.cu): whether they cover a call, the
// rows of their parts, and their launches (no_copies: the self-test's).
bool tc_covers(const ggrn_scan_call& c);
int64_t tc_part_rows(const ggrn_scan_call& c, int64_t longest);
int tc_run(const ggrn_scan_call& c, const Params& p, bool cut, cudaStream_t s,
           bool no_copies = false);

}  // namespace scan
}  // namespace ggrn
