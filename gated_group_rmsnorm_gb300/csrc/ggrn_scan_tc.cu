// ggrn_scan_tc.cu -- the state space scan of prompts in bf16 on the
// 5th-generation tensor cores.
//
// A chunk of Q = 128 tokens of one head is computed as products.  With
// l_t = dt_t a log2(e), L(i, j) = sum of l over (j, i], all powers base 2:
//   G    = C B^T                                   [Q, Q]
//   M_ij = G_ij dt_j 2^L(i, j) for j <= i, else 0  [Q, Q], rounded to bf16
//   dS^T = B^T (w X),  w_j = dt_j 2^L(Q-1, j)      [N, P], w X in three bf16 pieces
//   Y    = 2^L(i, -1) (C S^T) + M X + d X          [Q, P], S rounded to bf16
//   S'   = 2^L(Q-1, -1) S + dS                     f32, in registers
// The products accumulate in f32 in tensor memory.  Only the operands M and S
// are rounded to bf16 (2^-8 of each term of an output that is itself rounded
// to bf16: of the sum of the terms' sizes, which is more than the output's own
// rounding where they cancel); w X carries 24 bits, since its sums are the f32
// state that is returned.
//
// The decays of M come from sums inside blocks of 32 tokens: a row's factor
// for a whole column block is one exponential (row prefix + the blocks
// between), times a column's factor (suffix within its block, made once per
// chunk).  Every such factor is a power of a sum of l's between j and i, so
// none overflows where M does not; only the diagonal blocks take an
// exponential per element.  l is held to -256 and up: a product with a
// smaller one underflows in any case, and the prefix sums stay exact enough
// beside it.
//
// One CTA per part of a sequence and tile of a head's columns (80 at most), its
// warps specialised so that all stages of neighbouring chunks overlap:
//   M    4 warps   G out of tensor memory, decays applied, M back into it as
//                  the operand of M X
//   S    8 warps   S in registers; dS out of tensor memory, S into shared
//                  memory as the next chunk's operand
//   Y    4 warps   Y out of tensor memory, into X's place
//   1 warp         issues the products
//   1 warp         B and C (tensor-map copies, as soon as what read the ones
//                  before is done) and the decays
//   X    10 warps  (two for each 16 columns) X by asynchronous copies a chunk
//                  ahead, the pieces of w X, and Y from X's place to memory
// B and C lie in the 128-byte swizzled layout, which serves B as rows of state
// columns in G and as its transpose in dS; X, its pieces, S and Y in the
// 32-byte swizzled one, whose 16-column atoms fit any head size (the layout of
// an operand does not change a product's time).  Products are issued in the
// order C S, dS, M X, G of the next chunk (TWO_M: G before M X), which leaves
// every other stage the time of two products; C S has two places, so that it
// does not wait for the Y before (2 % in the first case below).  A product of
// M = 128, K = 16 takes 44 + N/2 clocks with A in shared memory and 11 + N/2
// with A in tensor memory or kept from the product before: hence M in tensor
// memory and each step of B^T kept for its three pieces.
//
// What bounds it: the chain of a chunk's stages, 2.5 us a chunk (64 columns
// 2.4, 80 columns 2.6; the products alone take 1.7), and about 10 us to start
// and end a launch.  4096 tokens of 96 heads of 80 x 128: 97 us, where the bytes
// take 22 and the products, at the rate of a large matrix product, 11; eight
// sequences of 2048 tokens, 80 heads of 64: 246 us.  One CTA per SM for all its
// parts, with no stop between them, was slower by a fifth a chunk, since the
// roles then have to keep more than their registers hold: 291 us for the eight
// sequences.  The
// stages' loops are kept small: unrolled, the eight of them ran out of the
// instruction cache (10 of 24 stall cycles an instruction) at a quarter of the
// speed.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "ggrn_optin.h"
#include "ggrn_scan.cuh"
#include "ggrn_umma.cuh"

namespace ggrn {
namespace scan {

namespace {

constexpr int kQ = 128;            // tokens of a chunk (the products' M)
constexpr int kMaxAtoms = 5;       // 16-column atoms of a tile of a head: 80 columns
constexpr uint32_t kFaultScanWait = 64u;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -256.0f;

// shared memory
constexpr uint32_t kRowsBytes = kQ * 128 * 2;      // B or C: 32 KB
constexpr uint32_t kAtomBytes = kQ * 16 * 2;       // one 16-column atom of X: 4 KB
constexpr uint32_t kDecayFloats = 5 * kQ + 8;      // pre, col, dt, w, row + block sums, decay
constexpr int kDecays = 3;                         // chunks of decays kept
// tensor memory columns
constexpr uint32_t kColG = 0, kColM = 128, kColDs = 192;

struct TcParams {
  Params p;
  unsigned int* fault;
  int tile;        // columns of a head per CTA, a multiple of 16 up to 80
  int xvec, ovec;  // bytes a copy of x (16 or 8) / a store of out (16 or 8) moves
};

// D (+)= A B with A [128, K] in tensor memory.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// Descriptors of operands stored with their K index across rows.  128-byte
// swizzle: 64 columns of a row, 8-row groups 1024 bytes apart (stride), the
// next 64 columns a whole tile further (leading offset).
__device__ __forceinline__ uint64_t desc_t128(uint32_t addr, uint32_t next) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(next >> 4) << 16) |
         (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// 32-byte swizzle: 16 columns of a row, 8-row groups of 256 bytes, the next 16
// columns an atom further.
__device__ __forceinline__ uint64_t desc_t32(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(kAtomBytes >> 4) << 16) | (uint64_t{256 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{6} << 61);
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;  // instruction descriptor bits

// Byte offset of 16-byte chunk `ch` (8 columns) of row r in 32-byte swizzled
// atoms.
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  return static_cast<uint32_t>((ch >> 1) * static_cast<int>(kAtomBytes) + r * 32 +
                               (((ch ^ (r >> 2)) & 1) << 4));
}
// The 16-byte chunks of a tile of `atoms` atoms, dealt to 64 threads an atom (4
// chunks each): eight lanes take four rows of an atom (its 128 bytes of shared
// memory, all banks), a warp the same rows of four atoms where there are as
// many, so that its global accesses are whole lines (16 rows of 32 bytes an
// instruction measured 94 clocks an instruction).  Chunk i of a thread is 32
// rows below its first one.
constexpr int kDealt = 4, kDealtRows = 32;
constexpr uint32_t kDealtBytes = kDealtRows * 32;
struct Deal {
  int row, col;
  uint32_t at;
  __device__ __forceinline__ Deal(int t, int atoms) {
    const int a = (t >> 3) % atoms, rows4 = (t >> 3) / atoms;
    row = 4 * rows4 + ((t & 7) >> 1);
    col = 16 * a + 8 * (t & 1);
    at = static_cast<uint32_t>(a * static_cast<int>(kAtomBytes) + row * 32 +
                               (((t ^ rows4) & 1) << 4));
  }
};

__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// The wait for two such loads: their registers pass through it, so that nothing
// that uses them can move before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]),
                 "+r"(a[7]), "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]),
                 "+r"(a[13]), "+r"(a[14]), "+r"(a[15])::"memory");
  asm volatile(""
               : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]),
                 "+r"(b[7]), "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]),
                 "+r"(b[13]), "+r"(b[14]), "+r"(b[15])::"memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
      :
      : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
using Bf = Elem<__nv_bfloat16>;

__device__ __forceinline__ F2 pair(uint32_t a, uint32_t b) {
  return pk2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint32_t bf16x2(F2 v) {
  float a, b;
  upk2(v, a, b);
  return Bf::pack2(a, b);
}
// the two halves of a word of bf16
__device__ __forceinline__ F2 wide(uint32_t u) {
  return pk2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// dt_of without branches or calls: softplus(v) = max(v, 0) + log1p(u), u =
// exp(-|v|), and log1p(u) = 2 atanh(r), r = u / (2 + u) <= 1/3, by its series up
// to r^15 (the next term is below 2^-27 of the first), so that a small dt keeps
// its relative accuracy: 2^-22 for u's exponential, |v| 2^-24 for its argument,
// 2^-22 for the quotient.
__device__ __forceinline__ float dt_of_fast(float raw, float bias, const Params& p) {
  float v = raw + bias;
  if (p.softplus) {
    const float u = ex2_approx(-kLog2e * fabsf(v));
    const float r = u * rcp_approx(2.0f + u), q = r * r;
    float t = 1.0f / 15;
    t = fmaf(t, q, 1.0f / 13);
    t = fmaf(t, q, 1.0f / 11);
    t = fmaf(t, q, 1.0f / 9);
    t = fmaf(t, q, 1.0f / 7);
    t = fmaf(t, q, 1.0f / 5);
    t = fmaf(t, q, 1.0f / 3);
    t = fmaf(t * q, r, r);
    v = fmaf(2.0f, t, v > 0.0f ? v : v != v ? v : 0.0f);
  }
  v = v < p.dt_min ? p.dt_min : v;
  return v > p.dt_max ? p.dt_max : v;
}

// The decays of one chunk, by one warp: dt of token 32 b + lane comes from
// `raw[b]` (tokens from `left` on count for nothing), goes through `s_dt`, and
// lane k takes tokens 4 k .. 4 k + 3, so that the blocks of 32 tokens are
// runs of 8 lanes.  pre: sums of l from the block's start, suf: to its end;
// before / after: sums of the blocks before and behind.  Returns the chunk's.
struct Decays {
  float dt[4], pre[4], suf[4];
  float block, before, after;
};
__device__ __forceinline__ float make_decays(const float (&raw)[4], int left, float bias, float a2,
                                             const Params& p, float* s_dt, Decays& d) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    s_dt[32 * b + lane] = 32 * b + lane < left ? dt_of_fast(raw[b], bias, p) : 0.0f;
  __syncwarp();
  const float4 v = *reinterpret_cast<const float4*>(s_dt + 4 * lane);
  d.dt[0] = v.x, d.dt[1] = v.y, d.dt[2] = v.z, d.dt[3] = v.w;
  float l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    l[k] = 4 * lane + k < left ? d.dt[k] * a2 : 0.0f;  // (not 0 times infinity)
    l[k] = l[k] < kMinLog ? kMinLog : l[k];
  }
  d.pre[0] = l[0];
  d.suf[3] = 0.0f;
#pragma unroll
  for (int k = 1; k < 4; ++k) d.pre[k] = d.pre[k - 1] + l[k];
#pragma unroll
  for (int k = 2; k >= 0; --k) d.suf[k] = d.suf[k + 1] + l[k + 1];
  // the lanes before and behind this one in its block
  float up = d.pre[3], down = d.pre[3];
  const int at = lane & 7;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, up, o, 8);
    const float w = __shfl_down_sync(0xffffffffu, down, o, 8);
    if (at >= o) up += u;
    if (at + o < 8) down += w;
  }
  d.block = __shfl_sync(0xffffffffu, up, 7, 8);
  up = __shfl_up_sync(0xffffffffu, up, 1, 8);
  down = __shfl_down_sync(0xffffffffu, down, 1, 8);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (at > 0) d.pre[k] += up;
    if (at < 7) d.suf[k] += down;
  }
  const float t0 = __shfl_sync(0xffffffffu, d.block, 0), t1 = __shfl_sync(0xffffffffu, d.block, 8),
              t2 = __shfl_sync(0xffffffffu, d.block, 16), t3 = __shfl_sync(0xffffffffu, d.block, 24);
  const int b = lane >> 3;
  d.before = b == 0 ? 0.0f : b == 1 ? t0 : b == 2 ? t0 + t1 : t0 + t1 + t2;
  d.after = b == 3 ? 0.0f : b == 2 ? t3 : b == 1 ? t3 + t2 : t3 + t2 + t1;
  return (t0 + t1) + (t2 + t3);
}
__device__ __forceinline__ void sts_f4(float* at, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(at) = make_float4(a, b, c, d);
}

// The three bf16 pieces of eight products w x, each piece what the ones before
// leave, cut off (not rounded: 8 bits each of 24).
// `odd` becomes NaN where a product is not finite.
__device__ __forceinline__ void pieces_of(const uint4& x, float w, uint4 (&u)[3], F2& odd) {
  const F2 ww = pk2(w, w), minus = pk2(-1.0f, -1.0f);
  uint32_t out[3][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    F2 v = mul2(wide((&x.x)[e]), ww);
    odd = fma2(v, 0, odd);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float a, b;
      upk2(v, a, b);
      const uint32_t ha = __float_as_uint(a), hb = __float_as_uint(b);
      out[k][e] = __byte_perm(ha, hb, 0x7632);
      if (k < 2) v = fma2(pair(ha & 0xffff0000u, hb & 0xffff0000u), minus, v);
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) u[k] = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
}

// Chunks with products that are not finite.  Such a product is its largest piece
// alone.  An x that is not finite is taken out of X, since M's zeros before its
// row would spread it over rows before its own; add_odd puts it back.  In its
// place stays the smallest normal number of its sign, which adds nothing to what
// add_odd makes infinite anyway: beside an infinite M (of an infinite dt) a zero
// there would be a NaN.
__device__ __noinline__ void odd_chunk(uint32_t x_at, uint32_t w_at, uint32_t x_bytes, float w) {
  for (int i = 0; i < 8; ++i) {
    unsigned short h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(x_at + 2 * i));
    const float v = w * __uint_as_float(static_cast<uint32_t>(h) << 16);
    if ((__float_as_uint(v) & 0x7f800000u) != 0x7f800000u) continue;
    const unsigned short top = static_cast<unsigned short>(v != v ? 0x7fc0 : __float_as_uint(v) >> 16);
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(w_at + 2 * i), "h"(top) : "memory");
    const unsigned short zero = 0;
    for (int k = 1; k < 3; ++k)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(w_at + k * x_bytes + 2 * i), "h"(zero) : "memory");
    const unsigned short least = (h & 0x8000) | 0x0080;
    if ((h & 0x7f80) == 0x7f80)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(x_at + 2 * i), "h"(least) : "memory");
  }
}
// What row i of a chunk's Y lacks for that: the terms of the x that are not
// finite, from the definition.  y: the chunk's place in shared memory, row: its
// first row, sd: its decays.
//
// The terms of one x and all n are infinities or NaN by the signs of B and C
// alone, so a row of x takes one pass over n for all its columns, and a column
// that is NaN takes no more.  (All roles wait meanwhile, for about a second at
// most.)  A chunk whose x are all NaN, or infinities with B and C of both signs,
// is done after its first row: 4096 tokens of 96 heads of 80 x 128 of NaN take
// 246 us.  The longest, infinities of one sign under B and C of one sign, takes
// 128 passes over n for its last row, 3.2 ms a chunk.
__device__ __noinline__ void add_odd(uint32_t y, const Params& p, int64_t row, int64_t hcol, int pw,
                                     int g, const float* sd, int i, float dskip) {
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + row * p.xs + hcol;
  const __nv_bfloat16* b =
      static_cast<const __nv_bfloat16*>(p.b) + row * p.bs + static_cast<int64_t>(g) * p.N;
  const __nv_bfloat16* c =
      static_cast<const __nv_bfloat16*>(p.c) + (row + i) * p.cs + static_cast<int64_t>(g) * p.N;
  auto at = [&](int col) { return y + chunk_at(i, col >> 3) + 2 * (col & 7); };
  auto load = [&](int col) {
    unsigned short h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at(col)));
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  };
  int open = 0;  // columns that are not NaN
  for (int col = 0; col < pw; ++col) open += load(col) == load(col);
#pragma unroll 1
  for (int j = 0; j <= i && open > 0; ++j) {
    // the terms of a row's +infinity; 0: not computed
    float terms = 0.0f;
#pragma unroll 1
    for (int col = 0; col < pw; ++col) {
      if (col % 4 == 0) {  // (rows are 8-byte aligned, pw a multiple of 4)
        const uint2 u = *reinterpret_cast<const uint2*>(x + j * p.xs + col);
        float v = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = e ? u.y : u.x;
          v += 0.0f * __uint_as_float(w << 16) + 0.0f * __uint_as_float(w & 0xffff0000u);
        }
        if (v == 0.0f) {
          col += 3;
          continue;
        }
      }
      const float v = Bf::load1(x + j * p.xs, col);
      if ((__float_as_uint(v) & 0x7f800000u) != 0x7f800000u) continue;
      float sum = load(col);
      if (sum != sum) continue;
      if (terms == 0.0f && v == v) {
        float l = sd[i] - sd[j], f = sd[2 * kQ + j];  // of one block: dt_j 2^(pre_i - pre_j)
        if (i >> 5 != j >> 5) {
          l = sd[i], f = sd[kQ + j];
          for (int k = (j >> 5) + 1; k < i >> 5; ++k) l += sd[5 * kQ + k];
        }
        const float m = f * ex2_approx(l) * INFINITY;
        for (int n = 0; n < p.N && terms == terms; ++n)
          terms += m * Bf::load1(b + j * p.bs, n) * Bf::load1(c, n);
      }
      sum += v != v ? v : v > 0.0f ? terms : -terms;
      if (j == i) sum += dskip * v;
      open -= sum != sum;
      const unsigned short h = static_cast<unsigned short>(Bf::pack2(sum, sum));
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at(col)), "h"(h) : "memory");
    }
  }
}

// `bytes` (16 or 8) from global to shared memory, of which the first `valid`
// are read and the rest zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Columns [col, col + 8) of a row of X (`src` points at them), zeros behind
// column pw and where the row is not `there` (nothing is read then; `base` is
// an address that could be); vec: rows are 16-byte aligned (else 8).
__device__ __forceinline__ void copy_x(uint32_t dst, const __nv_bfloat16* src,
                                       const __nv_bfloat16* base, int col, int pw, bool there,
                                       bool vec) {
  if (vec) {
    const bool v = there && col < pw;
    cp_async16(dst, v ? src : base, v ? 16 : 0);
  } else {
    const bool v0 = there && col < pw, v1 = there && col + 4 < pw;
    cp_async8(dst, v0 ? src : base, v0 ? 8 : 0);
    cp_async8(dst + 8, v1 ? src + 4 : base, v1 ? 8 : 0);
  }
}

// dS (+)= B^T [w X in pieces], smallest piece first; each step's B^T is kept
// for its three pieces.
__device__ __forceinline__ void issue_ds(uint32_t t_ds, uint64_t d_bt, uint64_t d_w, uint32_t piece,
                                         uint32_t idesc) {
#pragma unroll 1
  for (int k = 0; k < kQ / 16; ++k) {
    const uint64_t a = d_bt + k * (2048 >> 4), w = d_w + k * (512 >> 4);
    mma_bf16_keep<Keep::kFill>(t_ds, a, w + 2 * piece, idesc, k > 0);
    mma_bf16_keep<Keep::kUse>(t_ds, a, w + piece, idesc, true);
    mma_bf16_keep<Keep::kLast>(t_ds, a, w, idesc, true);
  }
}

// Bounded waits of a CTA, a whole warp at a time: a role whose wait runs out
// (after about a second) sets the CTA's flag and leaves its loop, the others
// follow, and the flag ends in the library's status word.  A try without a time
// hint suspends the warp for a while of the hardware's choosing; with a hint it
// is a sleep that ends late (450 clocks a wait that had nothing to wait for).
// The first try is inlined, the polling a function of its own: inlined at each
// of the waits it is larger than the instruction cache, and as one call with
// the first try it cost a fifth of the kernel's time.
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr long long kWaitClocks = 2000000000ll;
__device__ __noinline__ bool wait_poll(uint32_t bar, uint32_t parity, volatile uint32_t* flag) {
  const long long start = clock64();
  do {
    if (try_phase(bar, parity)) return true;
    if (*flag) return false;
  } while (clock64() - start < kWaitClocks);
  *flag = 1;
  return false;
}
struct Waits {
  volatile uint32_t* flag;
  __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
    parity &= 1u;
    if (__all_sync(0xffffffffu, try_phase(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_poll(bar, parity, flag)) != 0;
  }
};
// The end of a wait by a group of warps whose first one polled: its answer for
// all of them.  (Polled by every warp, the barriers slow each other and the
// rest of shared memory down.)
__device__ __forceinline__ bool group_sync(int id, int threads, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n"
      " barrier.cta.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

// D = A B with A [128, N] in rows of the 128-byte swizzle (K its columns), and
// B the same way, or (TB) with its K index across the rows of 32-byte atoms.
template <uint32_t TB>
__device__ __forceinline__ void issue_rows(uint32_t d, uint64_t da, uint64_t db, int ksteps,
                                           uint32_t idesc) {
#pragma unroll 1
  for (int k = 0; k < ksteps; k += 2) {
    mma_bf16(d, da, db, idesc, k > 0);
    if (k + 1 < ksteps) mma_bf16(d, da + 2, db + (TB ? 512 >> 4 : 2), idesc, true);
    // two steps of 32 bytes in a row, then the next 64 columns
    const uint32_t next = k & 2 ? (kRowsBytes / 2 - 64) >> 4 : 4;
    da += next;
    db += TB ? 2 * (512 >> 4) : next;
  }
}

// M of 16 columns of a block before the row's: G f c_j, f the row's factor and
// c_j the columns'.
__device__ __forceinline__ void decayed(const uint32_t (&g)[16], const float* cj, float f,
                                        uint32_t (&m)[8]) {
  const F2 ff = pk2(f, f);
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(cj + e);  // two pairs
    m[e / 2] = bf16x2(mul2(mul2(c.x, ff), pair(g[e], g[e + 1])));
    m[e / 2 + 1] = bf16x2(mul2(mul2(c.y, ff), pair(g[e + 2], g[e + 3])));
  }
}
// The same in the row's own block (whose decays start at `s`), of the columns
// up to `last`.
__device__ __forceinline__ void decayed_diagonal(const uint32_t (&g)[16], const float* s, float pre,
                                                 int last, uint32_t (&m)[8]) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 pj = *reinterpret_cast<const float2*>(s + e);
    const float2 dj = *reinterpret_cast<const float2*>(s + 2 * kQ + e);
    const float v0 = __uint_as_float(g[e]) * (dj.x * ex2_approx(pre - pj.x));
    const float v1 = __uint_as_float(g[e + 1]) * (dj.y * ex2_approx(pre - pj.y));
    m[e / 2] = Bf::pack2(e <= last ? v0 : 0.0f, e + 1 <= last ? v1 : 0.0f);
  }
}

// Arrive for a whole warp (each lane's earlier work included).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------------------
// k_scan_tc
// ---------------------------------------------------------------------------
constexpr int kMWarps = 4, kSWarps = 8, kYWarps = 4, kXWarps = 2 * kMaxAtoms;
constexpr int kWarpS = kMWarps, kWarpY = kWarpS + kSWarps, kWarpMma = kWarpY + kYWarps,
              kWarpDt = kWarpMma + 1, kWarpX = kWarpMma + 2;
constexpr int kMainThreads = (kWarpX + kXWarps) * 32;
constexpr int kSShare = kSWarps / 4;                      // warps on a quarter of the lanes
constexpr int kSAtoms = (kMaxAtoms + kSShare - 1) / kSShare;
// barriers, 8 bytes each; [2] and [3] by buffer
enum Bar {
  kBFull = 0,    // [2] B landed
  kBFree = 2,    // [2] B read by G and dS
  kCFull = 4,    // [2] C landed
  kCFree = 6,    // [2] C read by G and C S
  kYPut = 8,     // [2] Y in X's place
  kDtFull = 10,  // [3] decays made
  kDtFree = 13,  // [3] and read
  kTail = 16,    // B of a part's last, partial chunk landed
  kWFull = 17,   // X and w X written
  kGDone = 18,   // G computed
  kMFull = 19,   // M written, G read
  kDsDone = 20,  // dS and C S computed, w X and S read
  kSFull = 21,   // S written, dS read
  kYDone = 22,   // Y computed, M read
  kYRead = 23,   // Y read
  kBars = 24
};

// STATE_ONLY: the state a part adds from a zero start, and its decay (a cut
// sequence's parts but the last): dS and S alone; the warps of M and Y but the
// copying one have nothing to do.
// TWO_M: M has two places in tensor memory, and G of the next chunk goes before
// M X, so that M's warps need not wait for M X; there is room for that with
// tiles up to 64 columns (4096 tokens of 152 heads of 64: 89 us against 94; 80
// columns with it and one place for C S: 105 us against 95 in the case above).
// NO_COPIES: the self-test's, B and C never come, so that the waits for them run
// out.  (A form of its own: as a parameter of the others it cost 13 %.)
template <bool STATE_ONLY, bool TWO_M, bool NO_COPIES = false>
__global__ void __launch_bounds__(kMainThreads, 1)
    k_scan_tc(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
              const TcParams tp) {
  const Params& p = tp.p;
  pdl_wait();
  pdl_launch_dependents();
  const Part part = find_part<STATE_ONLY>(p.q, p.part, blockIdx.x);
  // (offsets that do not ascend may count more places than there are)
  if (part.seq < 0 ||
      (part.count > 1 && part.place + (STATE_ONLY ? 1 : 0) >= p.places))
    return;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  unsigned char* base = smem_raw + (base_u - raw_u);
  const int atoms = tp.tile / 16;
  const uint32_t x_bytes = atoms * kAtomBytes;
  const uint32_t sB = base_u, sC = sB + 2 * kRowsBytes;
  const uint32_t sW = sC + kRowsBytes;                   // three pieces of w X
  const uint32_t sX = sW + 3 * x_bytes;                  // [2]
  const uint32_t sS = sX + 2 * x_bytes;
  const uint32_t decay_off = sS + x_bytes - base_u;
  float* s_decay = reinterpret_cast<float*>(base + decay_off);
  const uint32_t bars_off = decay_off + kDecays * kDecayFloats * 4;
  volatile uint32_t* s_misc = reinterpret_cast<uint32_t*>(base + bars_off + 8 * kBars + 8);
  auto bar = [&](int i) { return base_u + bars_off + 8u * i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kBars) {
    const int i = tid;
    mbar_init(bar(i), i == kWFull                             ? 2 * atoms
                      : i == kMFull                           ? kMWarps
                      : i == kSFull                           ? kSWarps
                      : i == kYRead || i == kYPut || i == kYPut + 1 ? kYWarps
                      : i >= kDtFree && i < kDtFree + kDecays ? kSWarps + (STATE_ONLY ? 0 : kYWarps)
                                                              : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) s_misc[1] = 0, s_misc[2] = 0, s_misc[3] = 0;  // timeout; chunk + 1 with odd x, by buffer
  if (warp == kWarpMma) tmem_alloc(smem_u32(const_cast<uint32_t*>(s_misc)), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_misc[0];
  const uint32_t t_ds = tmem + kColDs, t_y2 = t_ds + tp.tile, t_y1 = t_y2 + tp.tile;  // y1: [2]
  const uint32_t t_m1 = tmem + (TWO_M ? kColDs + 4 * tp.tile : kColM);
  const int P = p.P, N = p.N;
  const int h = blockIdx.y, g = h / p.hpg;
  const int col0 = blockIdx.z * tp.tile;         // first column of the head here
  const int pw = min(tp.tile, P - col0);         // and how many
  const int64_t hcol = static_cast<int64_t>(h) * P + col0;
  const int rows = static_cast<int>(part.end - part.begin);
  const int chunks = (rows + kQ - 1) / kQ;
  const Waits wait = {s_misc + 1};
  // the state this part starts from (zeros without one) and the one it leaves
  const float* from = nullptr;
  float* to = nullptr;
  {
    const int64_t held = static_cast<int64_t>(P) * N, at = h * held + static_cast<int64_t>(col0) * N;
    const int64_t entry = seq_slot(p.q, part.seq);
    if (STATE_ONLY) {
      to = p.ws + (part.place + 1) * p.H * held + at;
    } else {
      if (part.count > 1) from = p.ws + part.place * p.H * held + at;
      else if (entry >= 0 && seq_resumes(p.q, part.seq)) from = p.state + entry * p.slot_stride + at;
      if (part.index == part.count - 1 && entry >= 0) to = p.state + entry * p.slot_stride + at;
    }
  }
  // Each phase of a barrier is waited for in turn: a parity tells a phase from
  // its neighbours only.  What may run ahead of a waiter by more is by buffer.

  if (warp == kWarpMma) {
    // ---- the products (the whole warp waits, one lane issues) ----
    const uint32_t id_g = idesc_bf16(128, 128);
    const uint32_t id_ds = idesc_bf16(128, tp.tile) | kTransA | kTransB;
    const uint32_t id_y = idesc_bf16(128, tp.tile) | kTransB;
    const uint64_t d_s = desc_t32(sS), d_w = desc_t32(sW), d_c = desc_sw128(sC);
    const uint32_t piece = x_bytes >> 4;
    const int ksteps = (N + 15) / 16;
    bool ok = true;
    // chunk c's C S, dS and M X, then the next one's G
#pragma unroll 1
    for (int c = STATE_ONLY ? 0 : -1; c < chunks; ++c) {
      const int n = c + 1, buf = n & 1;
      if (c >= 0) {
        // C S (S of the chunk before; dS read)
        if (!(ok = wait.warp(bar(kSFull), c))) break;
        if (!STATE_ONLY) {
          tc_fence_after();
          if (elect_one()) {
            issue_rows<kTransB>(t_y1 + (c & 1) * tp.tile, d_c, d_s, ksteps, id_y);
            mma_commit(bar(kCFree));
          }
          __syncwarp();
        } else if (!(ok = wait.warp(bar(kBFull + (c & 1)), c >> 1))) {
          break;
        }
        // dS
        if (!(ok = wait.warp(bar(kWFull), c))) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ds(t_ds, desc_t128(sB + (c & 1) * kRowsBytes, kRowsBytes / 2), d_w, piece, id_ds);
          mma_commit(bar(kDsDone));  // (and C S is: products end in order)
          mma_commit(bar(kBFree + (c & 1)));
        }
        __syncwarp();
        if (STATE_ONLY) continue;
        if (!(ok = wait.warp(bar(kMFull), c))) break;
      }
      // M X, and G of the next chunk: first where M has two places
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if ((step == 0) == TWO_M) {
          if (n >= chunks) continue;
          if (!(ok = wait.warp(bar(kBFull + buf), n >> 1) && wait.warp(bar(kCFull), n))) break;
          tc_fence_after();
          if (elect_one()) {
            issue_rows<0>(tmem + kColG, d_c, desc_sw128(sB + buf * kRowsBytes), ksteps, id_g);
            mma_commit(bar(kGDone));
          }
          __syncwarp();
        } else if (c >= 0) {
          // (Y of the chunk before read: C S has two places)
          if (c > 0 && !(ok = wait.warp(bar(kYRead), c - 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t d_x = desc_t32(sX + (c & 1) * x_bytes);
            const uint32_t t_m = TWO_M && (c & 1) ? t_m1 : tmem + kColM;
#pragma unroll 2
            for (int k = 0; k < kQ / 16; ++k)
              mma_bf16_ts(t_y2, t_m + 8 * k, d_x + k * (512 >> 4), id_y, k > 0);
            mma_commit(bar(kYDone));
          }
          __syncwarp();
        }
      }
      if (!ok) break;
    }
    // the last products are done before the tensor memory is freed
    if (STATE_ONLY && ok) ok = wait.warp(bar(kDsDone), chunks - 1);
    // no product may still run when the tensor memory is freed, and no copy be
    // on its way into shared memory: after a timeout, wait on a barrier of the
    // products' own, and as long again on one that nothing completes
    if (!ok) {
      if (elect_one()) {
        mbar_init(bar(kBars), 1);
        mma_commit(bar(kBars));
      }
      __syncwarp();
      mbar_wait(bar(kBars), 0);
      mbar_wait(bar(kBars), 1);
    }
  } else if (warp == kWarpDt) {
    // ---- B and C, as soon as what read the ones before is done, and the
    // decays of the chunk behind ----
    const int boxes = N > 64 ? 2 : 1;
    auto copy = [&](const CUtensorMap* map, uint32_t to_smem, int c, uint32_t full) {
      if (lane == 0 && !NO_COPIES) {
        mbar_expect_tx(full, boxes * (kRowsBytes / 2));
        for (int i = 0; i < boxes; ++i)
          tma_load_3d(to_smem + i * (kRowsBytes / 2), map, 64 * i, g,
                      static_cast<int>(part.begin) + c * kQ, full);
      }
      __syncwarp();
    };
    const float a2 = __ldg(p.a + h) * kLog2e;
    const float bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.0f;
    const __nv_bfloat16* dtp = static_cast<const __nv_bfloat16*>(p.dt) + part.begin * p.dts + h;
    float log_total = 0.0f;
    int slot = 0, use = 0;
#pragma unroll 1
    for (int c = -1; c < chunks; ++c) {
      float raw[4];  // of the next chunk
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = (c + 1) * kQ + 32 * b + lane;
        raw[b] = t < rows ? Bf::load1(dtp + t * p.dts, 0) : 0.0f;
      }
      // (the first chunk's copies before its decays, the others' behind them)
      const int n = c < 0 ? 0 : c;
      if (n < chunks && c != 0) {
        const int left = rows - n * kQ, buf = n & 1;
        const uint32_t b_at = sB + buf * kRowsBytes;
        if (n >= 2 && !wait.warp(bar(kBFree + buf), (n >> 1) - 1)) break;
        copy(&tm_b, b_at, n, bar(left < kQ ? static_cast<int>(kTail) : kBFull + buf));
        if (!STATE_ONLY) {
          if (n >= 1 && !wait.warp(bar(kCFree), n - 1)) break;
          copy(&tm_c, sC, n, bar(kCFull));
        }
      }
      if (c + 1 == chunks) break;
      if (use > 0 && !wait.warp(bar(kDtFree + slot), use - 1)) break;
      float* s = s_decay + slot * kDecayFloats;
      Decays d;
      const float total = make_decays(raw, rows - (c + 1) * kQ, bias, a2, p, s + 2 * kQ, d);
      float* t = s + 4 * lane;
      sts_f4(t, d.pre[0], d.pre[1], d.pre[2], d.pre[3]);
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = d.dt[k] * ex2_approx(d.suf[k]);
      sts_f4(t + kQ, f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = d.dt[k] * ex2_approx(d.suf[k] + d.after);
      sts_f4(t + 3 * kQ, f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = ex2_approx(d.before + d.pre[k]);
      sts_f4(t + 4 * kQ, f[0], f[1], f[2], f[3]);
      if ((lane & 7) == 0) s[5 * kQ + (lane >> 3)] = d.block;
      if (lane == 0) s[5 * kQ + 4] = ex2_approx(total);
      log_total += total;
      warp_arrive(bar(kDtFull + slot));
      if (++slot == kDecays) slot = 0, ++use;
    }
    if (STATE_ONLY && lane == 0 && blockIdx.z == 0)
      p.ws_decay[part.place * p.H + h] = ex2_approx(log_total);
    const int left = rows - (chunks - 1) * kQ;
    if (chunks > 0 && left < kQ && wait.warp(bar(kTail), 0)) {
      // rows of other sequences, or of none, count for nothing, whatever they
      // hold
      const int buf = (chunks - 1) & 1;
#pragma unroll 1
      for (int i = lane; i < (kQ - left) * 8; i += 32)
        for (int j = 0; j < boxes; ++j)
          sts16(sB + buf * kRowsBytes + j * (kRowsBytes / 2) + left * 128 + i * 16,
                make_uint4(0, 0, 0, 0));
      fence_async_smem();
      warp_arrive(bar(kBFull + buf));
    }
  } else if (warp >= kWarpX) {
    // ---- X in, a chunk ahead, and Y out, and the pieces of w X; a thread
    // reads, writes and stores its own chunks of a tile ----
    const int t = tid - kWarpX * 32, threads = 64 * atoms;
    if (t < threads) {
      const Deal deal(t, atoms);
      const int64_t first = part.begin + deal.row;
      const __nv_bfloat16* xp = static_cast<const __nv_bfloat16*>(p.x) + hcol + deal.col;
      __nv_bfloat16* op = static_cast<__nv_bfloat16*>(p.out) + hcol + deal.col;
      const __nv_bfloat16* x0 = static_cast<const __nv_bfloat16*>(p.x) + part.begin * p.xs + hcol;
      const bool cols = deal.col < pw, whole = tp.xvec == 16 && deal.col + 8 <= pw;
      int slot = 0, use = 0;
#pragma unroll 1
      for (int c = -1; c <= chunks; ++c) {
        if (c >= 0 && c < chunks) {
          bool ok = true;
          if (warp == kWarpX)
            ok = wait.warp(bar(kDtFull + slot), use) && (c == 0 || wait.warp(bar(kDsDone), c - 1));
          if (!group_sync(1, threads, ok)) break;
          const float* sw = s_decay + slot * kDecayFloats + 3 * kQ + deal.row;
          if (++slot == kDecays) slot = 0, ++use;
          cp_async_wait();
          const uint32_t x_at = sX + (c & 1) * x_bytes + deal.at, w_at = sW + deal.at;
          F2 odd = 0;
#pragma unroll 1
          for (int i = 0; i < kDealt; i += 2) {
            const uint32_t o = i * kDealtBytes;
            uint4 ua[3], ub[3];
            const uint4 xa = lds16(x_at + o), xb = lds16(x_at + o + kDealtBytes);
            pieces_of(xa, sw[i * kDealtRows], ua, odd);
            pieces_of(xb, sw[(i + 1) * kDealtRows], ub, odd);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              sts16(w_at + o + k * x_bytes, ua[k]);
              sts16(w_at + o + kDealtBytes + k * x_bytes, ub[k]);
            }
          }
          float odd0, odd1;
          upk2(odd, odd0, odd1);
          if (odd0 != odd0 || odd1 != odd1) {
            for (int i = 0; i < kDealt; ++i)
              odd_chunk(x_at + i * kDealtBytes, w_at + i * kDealtBytes, x_bytes,
                        sw[i * kDealtRows]);
            s_misc[2 + (c & 1)] = c + 1;
          }
          fence_async_smem();
          warp_arrive(bar(kWFull));
        }
        const int n = c + 1;  // the chunk to come into the place of n - 2
        const uint32_t x_at = sX + (n & 1) * x_bytes + deal.at;
        if (!STATE_ONLY && n >= 2) {
          const bool ok = warp != kWarpX || wait.warp(bar(kYPut + (n & 1)), (n >> 1) - 1);
          if (!group_sync(1, threads, ok)) break;
          const int left = rows - (n - 2) * kQ - deal.row;
          __nv_bfloat16* o = op + (first + (n - 2) * kQ) * p.os;
#pragma unroll 2
          for (int i = 0; i < kDealt; ++i, o += kDealtRows * p.os) {
            const uint4 v = lds16(x_at + i * kDealtBytes);
            if (i * kDealtRows < left && cols) {
              if (tp.ovec == 16) {
                *reinterpret_cast<uint4*>(o) = v;
              } else {
                *reinterpret_cast<uint2*>(o) = make_uint2(v.x, v.y);
                if (deal.col + 4 < pw) *reinterpret_cast<uint2*>(o + 4) = make_uint2(v.z, v.w);
              }
            }
          }
        }
        if (n < chunks) {
          const __nv_bfloat16* x = xp + (first + n * kQ) * p.xs;
          const int left = rows - n * kQ;
          if (left >= kQ && whole) {
#pragma unroll 2
            for (int i = 0; i < kDealt; ++i, x += kDealtRows * p.xs)
              cp_async16(x_at + i * kDealtBytes, x, 16);
          } else
#pragma unroll 1
          for (int i = 0; i < kDealt; ++i, x += kDealtRows * p.xs)
            copy_x(x_at + i * kDealtBytes, x, x0, deal.col, pw, deal.row + i * kDealtRows < left,
                   tp.xvec == 16);
        }
      }
      cp_async_wait();
    }
  } else if (warp < kWarpS) {
    // ---- M of rows 32 q + lane ----
    const int q = warp;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    int slot = 0, use = 0;
#pragma unroll 1
    for (int c = 0; c < (STATE_ONLY ? 0 : chunks); ++c) {
      // (G done: and the M before is read, by products issued earlier)
      bool ok = true;
      if (q == 0) ok = wait.warp(bar(kDtFull + slot), use) && wait.warp(bar(kGDone), c);
      if (!group_sync(2, kMWarps * 32, ok)) break;
      tc_fence_after();
      const float* sd = s_decay + slot * kDecayFloats;
      const float pre = sd[32 * q + lane];
      float between = pre;  // row prefix + the blocks between
#pragma unroll 1
      for (int blk = 3; blk >= 0; --blk) {
        const float* sj = sd + 32 * blk;
        const uint32_t t_g = tmem + lanes + kColG + 32 * blk;
        const uint32_t t_m = (TWO_M && (c & 1) ? t_m1 : tmem + kColM) + lanes + 16 * blk;
        uint32_t ga[16], gb[16], m[8];
        if (blk <= q) {
          tmem_ld16_nowait(t_g, ga);
          tmem_ld16_nowait(t_g + 16, gb);
        }
        if (blk < q) {
          const float f = ex2_approx(between);
          between += sj[5 * kQ - 31 * blk];  // the sum over this block
          tmem_ld_wait(ga, gb);
          decayed(ga, sj + kQ, f, m);
          tmem_st8(t_m, m);
          decayed(gb, sj + kQ + 16, f, m);
          tmem_st8(t_m + 8, m);
        } else if (blk == q) {
          tmem_ld_wait(ga, gb);
          decayed_diagonal(ga, sj, pre, lane, m);
          tmem_st8(t_m, m);
          decayed_diagonal(gb, sj + 16, pre, lane - 16, m);
          tmem_st8(t_m + 8, m);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = 0;
          tmem_st8(t_m, m);
          tmem_st8(t_m + 8, m);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(bar(kMFull));
      if (++slot == kDecays) slot = 0, ++use;
    }
  } else if (warp < kWarpY) {
    // ---- S: lanes 32 q.., atoms hf, hf + kSShare, .. ----
    const int q = warp & 3, hf = (warp - kWarpS) >> 2, n = 32 * q + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t at0 = sS + hf * kAtomBytes + chunk_at(n, 0);
    F2 s[kSAtoms][8];  // S^T: row n, columns 16 (hf + kSShare k) + 2 j and the next
    auto put = [&](int k) {  // atom k as the bf16 operand
#pragma unroll
      for (int ck = 0; ck < 2; ++ck)
        sts16((at0 + kSShare * k * kAtomBytes) ^ (ck << 4),
              make_uint4(bf16x2(s[k][4 * ck]), bf16x2(s[k][4 * ck + 1]), bf16x2(s[k][4 * ck + 2]),
                         bf16x2(s[k][4 * ck + 3])));
    };
    const int first = 16 * hf;  // column of the tile
#pragma unroll
    for (int k = 0; k < kSAtoms; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[k][j] = 0;
    if (from && n < N) {
      const float* f = from + first * N + n;
#pragma unroll
      for (int k = 0; k < kSAtoms; ++k, f += 16 * (kSShare - 1) * N)
#pragma unroll
        for (int j = 0; j < 8; ++j, f += 2 * N)
          if (first + 16 * kSShare * k + 2 * j < pw) s[k][j] = pk2(f[0], f[N]);  // (pw is even)
    }
    if (!STATE_ONLY) {
#pragma unroll
      for (int k = 0; k < kSAtoms; ++k)
        if (hf + kSShare * k < atoms) put(k);
      fence_async_smem();
    }
    warp_arrive(bar(kSFull));
    int slot = 0, use = 0;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      bool ok = true;
      if (warp == kWarpS) ok = wait.warp(bar(kDtFull + slot), use) && wait.warp(bar(kDsDone), c);
      if (!group_sync(3, kSWarps * 32, ok)) break;
      tc_fence_after();
      const float decay = s_decay[slot * kDecayFloats + 5 * kQ + 4];
      const F2 decay2 = pk2(decay, decay);
#pragma unroll
      for (int k = 0; k < kSAtoms; ++k) {
        const int a = hf + kSShare * k;
        if (a < atoms) {
          uint32_t r[16];
          tmem_ld16(t_ds + lanes + a * 16, r);
          if (n < N) {  // (rows behind N stay zeros: dS there is 0 times whatever w X is)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              s[k][j] = fma2(s[k][j], decay2, pair(r[2 * j], r[2 * j + 1]));
          }
          if (!STATE_ONLY) put(k);
        }
      }
      if (!STATE_ONLY) fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kSFull));
        mbar_arrive(bar(kDtFree + slot));
      }
      if (++slot == kDecays) slot = 0, ++use;
    }
    // the state after the part's last row
    if (to && n < N) {
      float* f = to + first * N + n;
#pragma unroll
      for (int k = 0; k < kSAtoms; ++k, f += 16 * (kSShare - 1) * N)
#pragma unroll
        for (int j = 0; j < 8; ++j, f += 2 * N)
          if (first + 16 * kSShare * k + 2 * j < pw) upk2(s[k][j], f[0], f[N]);
    }
  } else if (warp < kWarpMma) {
    // ---- Y: row 32 q + lane, into X's place ----
    const int q = warp & 3, i = 32 * q + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const float dskip = p.d ? __ldg(p.d + h) : 0.0f;
    const F2 skip2 = pk2(dskip, dskip);
    const uint32_t at0 = chunk_at(i, 0);
    int slot = 0, use = 0;
#pragma unroll 1
    for (int c = 0; c < (STATE_ONLY ? 0 : chunks); ++c) {
      bool ok = true;
      if (warp == kWarpY) ok = wait.warp(bar(kDtFull + slot), use) && wait.warp(bar(kYDone), c);
      if (!group_sync(4, kYWarps * 32, ok)) break;
      tc_fence_after();
      const float e = s_decay[slot * kDecayFloats + 4 * kQ + i];
      const F2 e2 = pk2(e, e);
      uint32_t at = sX + (c & 1) * x_bytes + at0;
#pragma unroll 1
      for (int a = 0; a < atoms; ++a, at += kAtomBytes) {
        uint32_t y1[16], y2[16];
        tmem_ld16_nowait(t_y1 + (c & 1) * tp.tile + lanes + a * 16, y1);
        tmem_ld16_nowait(t_y2 + lanes + a * 16, y2);
        uint4 xa = lds16(at), xb = lds16(at ^ 16);
        tmem_ld_wait(y1, y2);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          uint32_t& xw = j < 8 ? (&xa.x)[j / 2] : (&xb.x)[j / 2 - 4];
          xw = bf16x2(fma2(wide(xw), skip2,
                           fma2(pair(y1[j], y1[j + 1]), e2, pair(y2[j], y2[j + 1]))));
        }
        sts16(at, xa);
        sts16(at ^ 16, xb);
      }
      if (s_misc[2 + (c & 1)] == static_cast<uint32_t>(c + 1) && i < rows - c * kQ)
        add_odd(sX + (c & 1) * x_bytes, p, part.begin + c * kQ, hcol, pw, g,
                s_decay + slot * kDecayFloats, i, dskip);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kYRead));
        mbar_arrive(bar(kYPut + (c & 1)));
        mbar_arrive(bar(kDtFree + slot));
      }
      if (++slot == kDecays) slot = 0, ++use;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_misc[1]) atomicOr(tp.fault, kFaultScanWait);
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Times in chunks (see tc_part_rows).
constexpr double kStartChunks = 4.0, kStateShare = 0.6, kJoinChunks = 3.0;
uint32_t main_smem(int tile) {
  return 1024 + 3 * kRowsBytes + 6 * (tile / 16 * kAtomBytes) + kDecays * kDecayFloats * 4 +
         8 * kBars + 24;
}
int tile_of(int64_t P) {
  const int64_t tiles = (P + 16 * kMaxAtoms - 1) / (16 * kMaxAtoms);
  return static_cast<int>(((P + tiles - 1) / tiles + 15) / 16 * 16);
}

cudaError_t allow_smem() {
  const int bytes = static_cast<int>(main_smem(16 * kMaxAtoms));
  cudaError_t e = allow_shared_memory<k_scan_tc<false, false>>(bytes);
  if (e == cudaSuccess) e = allow_shared_memory<k_scan_tc<false, true>>(bytes);
  if (e == cudaSuccess) e = allow_shared_memory<k_scan_tc<true, false>>(bytes);
  if (e == cudaSuccess) e = allow_shared_memory<k_scan_tc<false, false, true>>(bytes);
  return e;
}

// [rows][groups][N] in boxes of 128 rows and 64 columns: columns behind N and
// rows behind the buffer read as zeros.
bool make_map(CUtensorMap* m, const void* ptr, int64_t N, int64_t groups, int64_t rows,
              int64_t stride) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(groups),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(N) * 2,
                                 static_cast<cuuint64_t>(rows > 1 ? stride : groups * N) * 2};
  const cuuint32_t box[3] = {64, 1, kQ};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

// bf16, state columns in whole 16-byte vectors and at most one tile, head
// columns in whole 8-byte ones, and rows aligned to those.
bool tc_covers(const ggrn_scan_call& c) {
  if (c.rows > INT32_MAX / 2 || c.b_row_stride >= int64_t{1} << 38 ||
      c.c_row_stride >= int64_t{1} << 38)
    return false;  // (what a tensor map holds)
  if (c.dtype != kBF16 || c.state_size % 8 != 0 || c.state_size > 128 || c.head_dim % 4 != 0)
    return false;
  const bool many = c.rows > 1;
  auto fits = [&](const void* ptr, int64_t stride, uintptr_t bytes) {
    return mixer::aligned_to(ptr, bytes) && (!many || stride * 2 % static_cast<int64_t>(bytes) == 0);
  };
  return fits(c.b, c.b_row_stride, 16) && fits(c.c, c.c_row_stride, 16) &&
         fits(c.x, c.x_row_stride, 8) && fits(c.out, c.out_row_stride, 8) &&
         (c.head_dim + tile_of(c.head_dim) - 1) / tile_of(c.head_dim) <= 65535;
}

// Rows of a part.  The launch's time goes by its waves of one CTA per SM, each
// as long as a part's chunks and about four more to start and end; a cut costs
// the state-only launch over the same chunks (a bit over half of a chunk's
// time) and the join.  The lengths behind cu_seqlens are not known here:
// sequences are taken for equally long, and where those stay whole a part is as
// long as the launch for them takes (and no less than twice their length): one
// sequence of that length may run beside the others.  3777 rows in 11 sequences
// of 0 to 918, 96 heads of 80 x 128: with parts of twice the mean, 50 of 190 us
// went into cutting two of them.  It is not free: CTAs start by part first and
// head second, so the long parts of the last heads start when the others are
// nearly done.  Counted in chunks as above, 12 sequences of 100 rows and one of
// 10000 behind them, 96 heads of 80, end after 143 (the longest first: 93; cut
// at twice the mean: 168).
int64_t tc_part_rows(const ggrn_scan_call& c, int64_t longest) {
  const int64_t tiles = (c.head_dim + tile_of(c.head_dim) - 1) / tile_of(c.head_dim);
  const int64_t heads = c.heads * tiles, sms = device_sms();
  const int64_t seqs = std::max<int64_t>(1, c.seqs);
  const int64_t most = std::max<int64_t>(1, (longest + kQ - 1) / kQ);
  const int64_t all =
      std::min(most, std::max<int64_t>(1, ((c.rows + seqs - 1) / seqs + kQ - 1) / kQ));
  auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
  int64_t best = all;
  double best_cost = 0.0;
  for (int64_t cuts = 1; cuts <= std::min<int64_t>(all, 64); ++cuts) {
    const int64_t k = (all + cuts - 1) / cuts;
    const int64_t parts = (all + k - 1) / k;
    double cost = static_cast<double>(waves(seqs * parts * heads)) * (k + kStartChunks);
    if (parts > 1)
      cost += static_cast<double>(waves(seqs * (parts - 1) * heads)) *
                  (kStateShare * k + kStartChunks) + kJoinChunks;
    if (cuts == 1 || cost < best_cost) {
      best = k;
      best_cost = cost;
    }
  }
  if (best < all) return best * kQ;
  const int64_t hidden = static_cast<int64_t>(best_cost - kStartChunks);
  return std::min(most, std::max(2 * all, hidden)) * kQ;
}

int tc_run(const ggrn_scan_call& c, const Params& p, bool cut, cudaStream_t s, bool no_copies) {
  TcParams tp;
  tp.p = p;
  tp.fault = device_fault_word();
  if (!tp.fault) return GGRN_ERR_CUDA;
  tp.tile = tile_of(p.P);
  tp.xvec = p.P % 8 == 0 && mixer::aligned_to(p.x, 16) && p.xs % 8 == 0 ? 16 : 8;
  tp.ovec = p.P % 8 == 0 && mixer::aligned_to(p.out, 16) && p.os % 8 == 0 ? 16 : 8;
  const cudaError_t e = allow_smem();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  CUtensorMap tm_b, tm_c;
  std::memset(&tm_b, 0, sizeof(tm_b));
  std::memset(&tm_c, 0, sizeof(tm_c));
  if (c.rows > 0 && (!make_map(&tm_b, c.b, c.state_size, c.groups, c.rows, c.b_row_stride) ||
                     !make_map(&tm_c, c.c, c.state_size, c.groups, c.rows, c.c_row_stride)))
    return GGRN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(p.parts), static_cast<unsigned>(p.H),
                  static_cast<unsigned>((p.P + tp.tile - 1) / tp.tile));
  if (cut) {
    int st = mixer::launch(k_scan_tc<true, false>, dim3(inner_parts(p), grid.y, grid.z), kMainThreads,
                           main_smem(tp.tile), s, tm_b, tm_c, tp);
    if (st != GGRN_OK) return st;
    st = launch_join(p, s);
    if (st != GGRN_OK) return st;
  }
  // (M's second place is behind the two of C S)
  const bool two_m = kColDs + 4 * tp.tile + 64 <= 512;
  if (no_copies)
    return mixer::launch(k_scan_tc<false, false, true>, grid, kMainThreads, main_smem(tp.tile), s,
                         tm_b, tm_c, tp);
  return mixer::launch(two_m ? k_scan_tc<false, true> : k_scan_tc<false, false>, grid, kMainThreads,
                       main_smem(tp.tile), s, tm_b, tm_c, tp);
}

}  // namespace scan
}  // namespace ggrn
