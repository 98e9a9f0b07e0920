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
// to bf16); w X carries 24 bits, since its sums are the f32 state that is
// returned.
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
// One CTA per part of a sequence and head (or tile of a head's columns):
// 16 warps share the elementwise work (X and its pieces into shared memory, G
// to M, S and Y out of tensor memory; a warp reads the 32 tensor-memory lanes
// that its number allows), one thread issues the products, one warp makes the
// decays a chunk ahead.  B and C come by asynchronous copies into the
// 128-byte swizzled layout, which serves B both as rows of the state columns
// (G) and as its transpose (dS); X, its pieces and S lie in the 32-byte
// swizzled layout, whose 16-column atoms fit any head size.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "ggrn_scan.cuh"
#include "ggrn_umma.cuh"

namespace ggrn {
namespace scan {

namespace {

constexpr int kQ = 128;            // tokens of a chunk (the products' M)
constexpr int kMaxAtoms = 6;       // 16-column atoms of a tile of a head: 96 columns
constexpr uint32_t kFaultScanWait = 64u;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -256.0f;

// shared memory
constexpr uint32_t kRowsBytes = kQ * 128 * 2;      // B or C: 32 KB
constexpr uint32_t kAtomBytes = kQ * 16 * 2;       // one 16-column atom of X: 4 KB
constexpr uint32_t kDecayFloats = 5 * kQ + 8;      // pre, col, dt, w, row + block sums, decay
// tensor memory columns (full kernel; the state-only one has dS at 0)
constexpr uint32_t kColG = 0, kColM = 128, kColDs = 192;

struct TcParams {
  Params p;
  unsigned int* fault;
  int tile;        // columns of a head per CTA, a multiple of 16 up to 96
  int xvec, ovec;  // 16-byte rows of x / out (else 8-byte)
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

// Byte offset of 16-byte chunk `ck` of row r of an atom.
__device__ __forceinline__ uint32_t atom_at(int r, int ck) {
  return (r >> 3) * 256 + (r & 7) * 32 + ((ck ^ ((r >> 2) & 1)) << 4);
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};"
      :
      : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(taddr)
      : "memory");
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
// 16 bytes to shared memory, zeros where !valid (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

using Bf = Elem<__nv_bfloat16>;

// WQ: warps on each quarter of the tensor-memory lanes.
template <int WQ, bool STATE_ONLY>
__global__ void __launch_bounds__((4 * WQ + 2) * 32, STATE_ONLY ? 2 : 1)
    k_scan_tc(const TcParams tp) {
  constexpr int NT = WQ * 128;                          // threads of the elementwise warps
  constexpr int AW = (kMaxAtoms + WQ - 1) / WQ;         // atoms of a warp
  constexpr int XI = (kMaxAtoms * 256 + NT - 1) / NT;   // 16-byte chunks of X of a thread
  const Params& p = tp.p;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_u = smem_u32(smem_raw);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  unsigned char* base = smem_raw + (base_u - raw_u);
  const int atoms = tp.tile / 16;
  const uint32_t x_bytes = atoms * kAtomBytes;
  const uint32_t sB = base_u, sC = sB + kRowsBytes;
  const uint32_t sW = sC + (STATE_ONLY ? 0 : kRowsBytes);  // three pieces of w X
  const uint32_t sX = sW + 3 * x_bytes, sS = sX + x_bytes;
  const uint32_t decay_off = (STATE_ONLY ? sX : sS + x_bytes) - base_u;
  float* s_decay = reinterpret_cast<float*>(base + decay_off);  // [2][kDecayFloats]
  const uint32_t bars = base_u + decay_off + 2 * kDecayFloats * 4;
  // a phase of each per chunk: B and C landed; X written (and everything of
  // the chunk before read); S written; M written; decays made; the products
  // done: G, dS with C S^T, all; and Y stored
  const uint32_t b_bc = bars, b_x = bars + 8, b_s = bars + 16, b_m = bars + 24, b_dt = bars + 32,
                 b_g = bars + 40, b_ds = bars + 48, b_y = bars + 56, b_e = bars + 64;
  volatile uint32_t* s_misc = reinterpret_cast<uint32_t*>(base + decay_off + 2 * kDecayFloats * 4 + 72);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    mbar_init(b_bc, NT);
    mbar_init(b_x, NT);
    mbar_init(b_s, NT);
    mbar_init(b_m, NT);
    mbar_init(b_dt, 32);
    mbar_init(b_g, 1);
    mbar_init(b_ds, 1);
    mbar_init(b_y, 1);
    mbar_init(b_e, NT);
    s_misc[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  constexpr uint32_t kTmemCols = STATE_ONLY ? 128 : 512;
  if (warp == 4 * WQ) tmem_alloc(smem_u32(const_cast<uint32_t*>(s_misc)), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_misc[0];
  const uint32_t t_ds = tmem + (STATE_ONLY ? 0 : kColDs);
  const uint32_t t_y1 = t_ds + tp.tile, t_y2 = t_y1 + tp.tile;
  pdl_wait();
  pdl_launch_dependents();

  const Part part = find_part(p.q, p.part, blockIdx.x);
  const int P = p.P, N = p.N;
  const int h = blockIdx.y;
  const int col0 = blockIdx.z * tp.tile;         // first column of the head here
  bool run = part.seq >= 0 && !(STATE_ONLY && part.index == part.count - 1) &&
             !(part.count > 1 && part.place + (STATE_ONLY ? 1 : 0) >= p.places);
  const int64_t rows = run ? part.end - part.begin : 0;
  const int chunks = static_cast<int>((rows + kQ - 1) / kQ);
  auto fail = [&]() {
    s_misc[1] = 1;
    atomicOr(tp.fault, kFaultScanWait);
  };
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!s_misc[1] && mbar_wait(bar, parity & 1u)) return true;
    if (!s_misc[1]) fail();
    return false;
  };

  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };

  if (!run) {
    // nothing: fall through to the end
  } else if (warp == 4 * WQ) {
    // ---- the products ----
    if (lane == 0) {
      const uint32_t id_g = idesc_bf16(128, 128);
      const uint32_t id_ds = idesc_bf16(128, tp.tile) | kTransA | kTransB;
      const uint32_t id_y = idesc_bf16(128, tp.tile) | kTransB;
      const uint64_t d_b = desc_sw128(sB), d_c = desc_sw128(sC);
      const uint64_t d_bt = desc_t128(sB, kRowsBytes / 2);
      const uint64_t d_x = desc_t32(sX), d_s = desc_t32(sS);
      const int ksteps = (N + 15) / 16;
      // step k of 16 along the columns of a 128-byte swizzled tile
      auto kk = [](int k) { return static_cast<uint64_t>((k >> 2) * (kRowsBytes / 2) + (k & 3) * 32) >> 4; };
      int c = 0;
      for (; c < chunks; ++c) {
        if (!wait(b_bc, c)) break;
        tc_fence_after();
        if (!STATE_ONLY) {
          for (int k = 0; k < ksteps; ++k)
            mma_bf16(tmem + kColG, d_c + kk(k), d_b + kk(k), id_g, k > 0);
          mma_commit(b_g);
        }
        if (!wait(b_x, c)) break;
        tc_fence_after();
#pragma unroll
        for (int piece = 2; piece >= 0; --piece) {
          const uint64_t d_w = desc_t32(sW + piece * x_bytes);
#pragma unroll
          for (int k = 0; k < kQ / 16; ++k)
            mma_bf16(t_ds, d_bt + k * (2048 >> 4), d_w + k * (512 >> 4), id_ds,
                     piece < 2 || k > 0);
        }
        if (!STATE_ONLY) {
          if (!wait(b_s, c)) break;
          tc_fence_after();
          for (int k = 0; k < ksteps; ++k)
            mma_bf16(t_y1, d_c + kk(k), d_s + k * (512 >> 4), id_y, k > 0);
        }
        mma_commit(b_ds);
        if (!STATE_ONLY) {
          if (!wait(b_m, c)) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kQ / 16; ++k)
            mma_bf16_ts(t_y2, tmem + kColM + 8 * k, d_x + k * (512 >> 4), id_y, k > 0);
          mma_commit(b_y);
        }
      }
      // no product may still run when the tensor memory is freed
      if (c < chunks) {
        mma_commit(b_y);
        for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait(b_y, c & 1u); ++i) {
        }
      }
    }
  } else if (warp == 4 * WQ + 1) {
    // ---- the decays, a chunk ahead ----
    const float a2 = __ldg(p.a + h) * kLog2e;
    const float bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.0f;
    const __nv_bfloat16* dtp = static_cast<const __nv_bfloat16*>(p.dt) + part.begin * p.dts + h;
    float raw[4];
    auto fetch = [&](int c) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int64_t t = static_cast<int64_t>(c) * kQ + 32 * b + lane;
        raw[b] = t < rows ? Bf::load1(dtp + t * p.dts, 0) : 0.0f;
      }
    };
    fetch(0);
    float log_total = 0.0f;
    for (int c = 0; c < chunks; ++c) {
      float pre[4], suf[4], tot[4], dt[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const bool valid = static_cast<int64_t>(c) * kQ + 32 * b + lane < rows;
        dt[b] = valid ? dt_of(raw[b], bias, p) : 0.0f;
        float l = valid ? dt[b] * a2 : 0.0f;
        l = l < kMinLog ? kMinLog : l;
        pre[b] = l;
        suf[b] = __shfl_down_sync(0xffffffffu, l, 1);
        if (lane == 31) suf[b] = 0.0f;
      }
      if (c + 1 < chunks) fetch(c + 1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float u = __shfl_up_sync(0xffffffffu, pre[b], o);
          const float d = __shfl_down_sync(0xffffffffu, suf[b], o);
          if (lane >= o) pre[b] += u;
          if (lane + o < 32) suf[b] += d;
        }
#pragma unroll
      for (int b = 0; b < 4; ++b) tot[b] = __shfl_sync(0xffffffffu, pre[b], 31);
      // this half of the decays was last read for chunk c - 2
      if (c >= 2 && !warp_wait(b_x, c - 1)) break;
      float* s = s_decay + (c & 1) * kDecayFloats;
      float before = 0.0f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float after = 0.0f;
#pragma unroll
        for (int k = 3; k > b; --k) after += tot[k];
        const int t = 32 * b + lane;
        s[t] = pre[b];
        s[kQ + t] = dt[b] * ex2_approx(suf[b]);
        s[2 * kQ + t] = dt[b];
        s[3 * kQ + t] = dt[b] * ex2_approx(suf[b] + after);
        s[4 * kQ + t] = ex2_approx(before + pre[b]);
        before += tot[b];
        if (lane == 0) s[5 * kQ + b] = tot[b];
      }
      if (lane == 0) s[5 * kQ + 4] = ex2_approx(before);
      log_total += before;
      mbar_arrive(b_dt);
    }
    if (STATE_ONLY && lane == 0 && blockIdx.z == 0)
      p.ws_decay[part.place * p.H + h] = ex2_approx(log_total);
  } else {
    // ---- the elementwise warps ----
    const int q = warp & 3, hf = warp >> 2;  // lanes 32 q.. of tensor memory; share of the columns
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    const int g = h / p.hpg;
    const int64_t hcol = static_cast<int64_t>(h) * P + col0;
    const int pw = min(tp.tile, P - col0);   // columns here
    const __nv_bfloat16* xg = static_cast<const __nv_bfloat16*>(p.x) + part.begin * p.xs + hcol;
    const __nv_bfloat16* bg =
        static_cast<const __nv_bfloat16*>(p.b) + part.begin * p.bs + static_cast<int64_t>(g) * N;
    const __nv_bfloat16* cg =
        static_cast<const __nv_bfloat16*>(p.c) + part.begin * p.cs + static_cast<int64_t>(g) * N;
    __nv_bfloat16* og = static_cast<__nv_bfloat16*>(p.out) + part.begin * p.os + hcol;
    const float dskip = p.d ? __ldg(p.d + h) : 0.0f;
    const int64_t slot = seq_slot(p.q, part.seq);

    auto load_bc = [&](int c) {
#pragma unroll
      for (int it = 0; it < 2048 / NT; ++it) {
        const int id = it * NT + tid, r = id >> 4, ch = id & 15;
        const int64_t t = static_cast<int64_t>(c) * kQ + r;
        const bool valid = t < rows && ch * 8 < N;
        const uint32_t at = (ch >> 3) * (kRowsBytes / 2) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
        cp_async16(sB + at, valid ? bg + t * p.bs + ch * 8 : bg, valid);
        if (!STATE_ONLY) cp_async16(sC + at, valid ? cg + t * p.cs + ch * 8 : cg, valid);
      }
    };
    uint4 xr[XI];
    auto fetch_x = [&](int c) {
#pragma unroll
      for (int it = 0; it < XI; ++it) {
        const int id = it * NT + tid;
        const int r = (id & 255) >> 1, col = (id >> 8) * 16 + (id & 1) * 8;
        const int64_t t = static_cast<int64_t>(c) * kQ + r;
        xr[it] = make_uint4(0, 0, 0, 0);
        if (t < rows && col < pw) {
          const __nv_bfloat16* src = xg + t * p.xs + col;
          if (tp.xvec) {
            xr[it] = ld_stream(src);
          } else {
            const uint2 lo = __ldg(reinterpret_cast<const uint2*>(src));
            xr[it].x = lo.x, xr[it].y = lo.y;
            if (col + 4 < pw) {
              const uint2 hi = __ldg(reinterpret_cast<const uint2*>(src + 4));
              xr[it].z = hi.x, xr[it].w = hi.y;
            }
          }
        }
      }
    };
    if (chunks > 0) {
      load_bc(0);
      fetch_x(0);
    }
    // the state: lane n = 32 q + lane of S^T, columns 16 (hf + WQ k) + j
    float s[AW][16];
    const int n = 32 * q + lane;
    const int64_t PN = static_cast<int64_t>(P) * N;
    const float* from = nullptr;
    if (!STATE_ONLY) {
      if (part.count > 1) from = p.ws + (part.place * p.H + h) * PN;
      else if (slot >= 0 && seq_resumes(p.q, part.seq)) from = p.state + slot * p.slot_stride + h * PN;
    }
    auto put_state = [&](int k) {  // its atom k as the bf16 operand
      float v[8];
#pragma unroll
      for (int ck = 0; ck < 2; ++ck) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s[k][8 * ck + j];
        sts16(sS + (hf + WQ * k) * kAtomBytes + atom_at(n, ck), Bf::pack(v));
      }
    };
#pragma unroll
    for (int k = 0; k < AW; ++k) {
      const int a = hf + WQ * k;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int col = a * 16 + j;
        s[k][j] = from && n < N && a < atoms && col < pw
                      ? from[static_cast<int64_t>(col0 + col) * N + n] : 0.0f;
      }
      if (!STATE_ONLY && a < atoms) put_state(k);
    }
    if (!STATE_ONLY) {
      fence_async_smem();
      mbar_arrive(b_s);
    }

    for (int c = 0; c < chunks; ++c) {
      const float* sd = s_decay + (c & 1) * kDecayFloats;
      cp_async_wait();
      fence_async_smem();
      mbar_arrive(b_bc);
      // X and the pieces of w X
      if (!warp_wait(b_dt, c)) break;
      // (other warps may still read X of the chunk before)
      if (!STATE_ONLY && c > 0 && !warp_wait(b_e, c - 1)) break;
#pragma unroll
      for (int it = 0; it < XI; ++it) {
        const int id = it * NT + tid;
        if (id < atoms * 256) {
          const int r = (id & 255) >> 1;
          const uint32_t at = (id >> 8) * kAtomBytes + atom_at(r, id & 1);
          const float w = sd[3 * kQ + r];
          float v[8], hi[8];
          Bf::unpack(xr[it], v);
#pragma unroll
          for (int e = 0; e < 8; e += 2) mul2(v[e], v[e + 1], v[e], v[e + 1], w, w);
          if (!STATE_ONLY) sts16(sX + at, xr[it]);
#pragma unroll
          for (int piece = 0; piece < 3; ++piece) {
            const uint4 u = Bf::pack(v);
            sts16(sW + piece * x_bytes + at, u);
            if (piece < 2) {
              Bf::unpack(u, hi);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] -= hi[e];
            }
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(b_x);
      if (c + 1 < chunks) fetch_x(c + 1);

      if constexpr (!STATE_ONLY) {
        // M of rows 32 q.. and columns 32 hf.. (WQ == 4)
        uint32_t m[16];
        if (hf <= q) {
          if (!warp_wait(b_g, c)) break;
          tc_fence_after();
          uint32_t gr[32];
          tmem_ld32_nowait(tmem + lanes + kColG + 32 * hf, gr);
          const float pre = sd[32 * q + lane];
          if (hf < q) {
            float between = pre;
            for (int b = hf + 1; b < q; ++b) between += sd[5 * kQ + b];
            const float f = ex2_approx(between);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 cf = *reinterpret_cast<const float4*>(sd + kQ + 32 * hf + j);
              float v0, v1, v2, v3;
              mul2(v0, v1, cf.x, cf.y, f, f);
              mul2(v2, v3, cf.z, cf.w, f, f);
              mul2(v0, v1, v0, v1, __uint_as_float(gr[j]), __uint_as_float(gr[j + 1]));
              mul2(v2, v3, v2, v3, __uint_as_float(gr[j + 2]), __uint_as_float(gr[j + 3]));
              m[j / 2] = Bf::pack2(v0, v1);
              m[j / 2 + 1] = Bf::pack2(v2, v3);
            }
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 pj = *reinterpret_cast<const float4*>(sd + 32 * hf + j);
              const float4 dj = *reinterpret_cast<const float4*>(sd + 2 * kQ + 32 * hf + j);
              const float v0 = __uint_as_float(gr[j]) * (dj.x * ex2_approx(pre - pj.x));
              const float v1 = __uint_as_float(gr[j + 1]) * (dj.y * ex2_approx(pre - pj.y));
              const float v2 = __uint_as_float(gr[j + 2]) * (dj.z * ex2_approx(pre - pj.z));
              const float v3 = __uint_as_float(gr[j + 3]) * (dj.w * ex2_approx(pre - pj.w));
              m[j / 2] = Bf::pack2(j <= lane ? v0 : 0.0f, j + 1 <= lane ? v1 : 0.0f);
              m[j / 2 + 1] = Bf::pack2(j + 2 <= lane ? v2 : 0.0f, j + 3 <= lane ? v3 : 0.0f);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) m[j] = 0;
        }
        tmem_st16(tmem + lanes + kColM + 16 * hf, m);
        tc_fence_before();
        mbar_arrive(b_m);
      }

      // S: B and C are read, the next ones may come
      if (!warp_wait(b_ds, c)) break;
      tc_fence_after();
      if (c + 1 < chunks) load_bc(c + 1);
      const float decay = sd[5 * kQ + 4];
#pragma unroll
      for (int k = 0; k < AW; ++k) {
        const int a = hf + WQ * k;
        if (a < atoms) {
          uint32_t r[16];
          tmem_ld16(t_ds + lanes + a * 16, r);
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            fma2(s[k][j], s[k][j + 1], s[k][j], s[k][j + 1], decay, decay, __uint_as_float(r[j]),
                 __uint_as_float(r[j + 1]));
          if (!STATE_ONLY) put_state(k);
        }
      }
      tc_fence_before();
      if constexpr (!STATE_ONLY) {
        fence_async_smem();
        mbar_arrive(b_s);
        // Y
        if (!warp_wait(b_y, c)) break;
        tc_fence_after();
        const int i = 32 * q + lane;
        const int64_t t = static_cast<int64_t>(c) * kQ + i;
        const float e = sd[4 * kQ + i];
#pragma unroll
        for (int k = 0; k < AW; ++k) {
          const int a = hf + WQ * k;
          if (a >= atoms) continue;
          uint32_t y1[16], y2[16];
          tmem_ld16(t_y1 + lanes + a * 16, y1);
          tmem_ld16(t_y2 + lanes + a * 16, y2);
#pragma unroll
          for (int ck = 0; ck < 2; ++ck) {
            float xv[8], y[8];
            Bf::unpack(lds16(sX + a * kAtomBytes + atom_at(i, ck)), xv);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              fma2(y[j], y[j + 1], __uint_as_float(y1[8 * ck + j]),
                   __uint_as_float(y1[8 * ck + j + 1]), e, e, __uint_as_float(y2[8 * ck + j]),
                   __uint_as_float(y2[8 * ck + j + 1]));
              fma2(y[j], y[j + 1], xv[j], xv[j + 1], dskip, dskip, y[j], y[j + 1]);
            }
            const int col = a * 16 + ck * 8;
            if (t < rows && col < pw) {
              const uint4 v = Bf::pack(y);
              __nv_bfloat16* o = og + t * p.os + col;
              if (tp.ovec) {
                *reinterpret_cast<uint4*>(o) = v;
              } else {
                *reinterpret_cast<uint2*>(o) = make_uint2(v.x, v.y);
                if (col + 4 < pw) *reinterpret_cast<uint2*>(o + 4) = make_uint2(v.z, v.w);
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(b_e);
      }
    }
    cp_async_wait();

    // the state after the part's last row
    float* to = nullptr;
    if (STATE_ONLY) to = p.ws + ((part.place + 1) * p.H + h) * PN;
    else if (part.index == part.count - 1 && slot >= 0) to = p.state + slot * p.slot_stride + h * PN;
    if (to && n < N) {
#pragma unroll
      for (int k = 0; k < AW; ++k)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int col = (hf + WQ * k) * 16 + j;
          if (hf + WQ * k < atoms && col < pw) to[static_cast<int64_t>(col0 + col) * N + n] = s[k][j];
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * WQ) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

uint32_t smem_bytes(int tile, bool state_only) {
  const uint32_t x = tile / 16 * kAtomBytes;
  return 1024 + (state_only ? kRowsBytes + 3 * x : 2 * kRowsBytes + 5 * x) +
         2 * kDecayFloats * 4 + 72 + 8;
}

int tile_of(int64_t P) {
  const int64_t tiles = (P + 16 * kMaxAtoms - 1) / (16 * kMaxAtoms);
  return static_cast<int>(((P + tiles - 1) / tiles + 15) / 16 * 16);
}

constexpr int kMainWq = 4, kStateWq = 2;

cudaError_t allow_smem() {
  static std::once_flag once;
  static cudaError_t err = cudaSuccess;
  std::call_once(once, [] {
    err = cudaFuncSetAttribute(k_scan_tc<kMainWq, false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem_bytes(16 * kMaxAtoms, false)));
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(k_scan_tc<kStateWq, true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem_bytes(16 * kMaxAtoms, true)));
  });
  return err;
}

}  // namespace

// bf16, state columns in whole 16-byte vectors and at most one tile, head
// columns in whole 8-byte ones, and rows aligned to those.
bool tc_covers(const ggrn_scan_call& c) {
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
// as long as a part's chunks; a cut costs the state-only launch over the same
// chunks (about half of a chunk's time, two CTAs per SM) and the join.  The
// lengths behind cu_seqlens are not known here: rows and sequences stand for
// the number of parts.
int64_t tc_part_rows(const ggrn_scan_call& c, int64_t longest) {
  const int64_t tiles = (c.head_dim + tile_of(c.head_dim) - 1) / tile_of(c.head_dim);
  const int64_t heads = c.heads * tiles, sms = device_sms();
  const int64_t all = std::max<int64_t>(1, (longest + kQ - 1) / kQ);
  const int64_t seqs = std::max<int64_t>(1, c.seqs);
  auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
  int64_t best = all;
  double best_cost = 0.0;
  // parts of a whole number of chunks, as many as make a difference
  for (int64_t cuts = 1; cuts <= std::min<int64_t>(all, 64); ++cuts) {
    const int64_t k = (all + cuts - 1) / cuts;
    const int64_t parts = c.cu_seqlens ? (c.rows + k * kQ - 1) / (k * kQ) + (seqs - 1)
                                       : seqs * ((all + k - 1) / k);
    double cost = static_cast<double>(waves(parts * heads)) * (k + 1.0);
    if (k < all) {
      const int64_t inner = std::max<int64_t>(1, parts - seqs);
      cost += 0.5 * static_cast<double>(waves((inner * heads + 1) / 2)) * (k + 1.0) + 2.0;
    }
    if (cuts == 1 || cost < best_cost) {
      best = k;
      best_cost = cost;
    }
  }
  return best * kQ;
}

int tc_run(const ggrn_scan_call& c, const Params& p, bool cut, cudaStream_t s) {
  TcParams tp;
  tp.p = p;
  tp.fault = device_fault_word();
  if (!tp.fault) return GGRN_ERR_CUDA;
  tp.tile = tile_of(p.P);
  tp.xvec = p.P % 8 == 0 && mixer::aligned_to(p.x, 16) && p.xs % 8 == 0;
  tp.ovec = p.P % 8 == 0 && mixer::aligned_to(p.out, 16) && p.os % 8 == 0;
  const cudaError_t e = allow_smem();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  const dim3 grid(static_cast<unsigned>(p.parts), static_cast<unsigned>(p.H),
                  static_cast<unsigned>((p.P + tp.tile - 1) / tp.tile));
  if (cut) {
    int st = mixer::launch(k_scan_tc<kStateWq, true>, grid, (4 * kStateWq + 2) * 32,
                           smem_bytes(tp.tile, true), s, tp);
    if (st != GGRN_OK) return st;
    st = launch_join(p, s);
    if (st != GGRN_OK) return st;
  }
  return mixer::launch(k_scan_tc<kMainWq, false>, grid, (4 * kMainWq + 2) * 32,
                       smem_bytes(tp.tile, false), s, tp);
}

}  // namespace scan
}  // namespace ggrn
