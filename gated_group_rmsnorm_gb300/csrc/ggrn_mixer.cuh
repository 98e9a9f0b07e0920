// ggrn_mixer.cuh -- what the mixer's convolution and scan kernels share: the
// ranges of packed sequences, their entries in a state pool, and the host's
// argument checks.
#pragma once

#include <initializer_list>

#include "../../include/ggrn.h"
#include "ggrn_kernels.cuh"

namespace ggrn {

// ---------------------------------------------------------------------------
// Two f32 in a register pair (see fma2 in ggrn_kernels.cuh): values that stay
// pairs from their load to their store need no moves between registers.
// ---------------------------------------------------------------------------
using Two = unsigned long long;  // two f32
__device__ __forceinline__ Two join(float a, float b) {
  return __builtin_bit_cast(Two, make_float2(a, b));
}
__device__ __forceinline__ void split(Two v, float& a, float& b) {
  const float2 f = __builtin_bit_cast(float2, v);
  a = f.x, b = f.y;
}
__device__ __forceinline__ float2 halves(Two v) { return __builtin_bit_cast(float2, v); }
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
  return __builtin_bit_cast(Two, __ffma2_rn(halves(a), halves(b), halves(c)));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  return __builtin_bit_cast(Two, __fmul2_rn(halves(a), halves(b)));
}
__device__ __forceinline__ Two add(Two a, Two b) {
  return __builtin_bit_cast(Two, __fadd2_rn(halves(a), halves(b)));
}
// f of each half.
template <typename F>
__device__ __forceinline__ Two each(Two a, F f) {
  float x, y;
  split(a, x, y);
  return join(f(x), f(y));
}
// A constant that stays in registers: made once, where it is written, and not
// again at each use (which takes two moves).
__device__ __forceinline__ Two held(float v) {
  Two r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
// The sequences of a call (see ggrn.h): cu == NULL means seqs equal ones.
struct Seqs {
  const int32_t* cu;
  const int32_t* slots;
  const uint8_t* resume;
  int64_t rows;
  int64_t seqs;
  int64_t each;         // rows of a sequence without cu
  int64_t state_slots;  // 0: no pool
};

// Rows [begin, end) of sequence i, clamped into [0, rows] so that no offset
// read from the device can lead outside the buffers.
__device__ __forceinline__ void seq_range(const Seqs& q, int64_t i, int64_t& begin, int64_t& end) {
  if (q.cu) {
    const int64_t b = __ldg(q.cu + i), e = __ldg(q.cu + i + 1);
    begin = b < 0 ? 0 : (b > q.rows ? q.rows : b);
    end = e < begin ? begin : (e > q.rows ? q.rows : e);
  } else {
    begin = i * q.each;
    end = begin + q.each;
  }
}

// Pool entry of sequence i, or -1.
__device__ __forceinline__ int64_t seq_slot(const Seqs& q, int64_t i) {
  if (q.state_slots == 0) return -1;
  const int64_t s = q.slots ? __ldg(q.slots + i) : i;
  return s >= 0 && s < q.state_slots ? s : -1;
}
__device__ __forceinline__ bool seq_resumes(const Seqs& q, int64_t i) {
  return q.resume && __ldg(q.resume + i) != 0;
}

// A sequence of n rows is cut into max(1, ceil(n / part)) parts of `part`
// rows; the parts of all sequences are numbered in order, at most
// rows / part + seqs of them.  The parts of sequences with more than one are
// numbered again, by themselves (their places, at most 2 rows / part: such a
// sequence is longer than a part).
struct Part {
  int64_t seq = -1;            // -1: the number is behind the last part
  int64_t begin = 0, end = 0;  // rows
  int64_t index = 0, count = 1;  // this part among those of its sequence
  int64_t place = 0;           // of a sequence with more than one part
};
// (With cu, and wherever sequences are cut, rows fit 32 bits: the host checks.)
__device__ __forceinline__ int64_t parts_of(int64_t n, int64_t part) {
  return n <= part ? 1
                   : (static_cast<uint32_t>(n) + static_cast<uint32_t>(part) - 1) /
                         static_cast<uint32_t>(part);
}
// Parts, or (INNER) parts but the last, in the low word and places in the high
// word, of a sequence of n rows.
template <bool INNER = false>
__device__ __forceinline__ uint64_t part_counts(int64_t n, int64_t part) {
  const uint64_t k = static_cast<uint64_t>(parts_of(n, part));
  return (INNER ? k - 1 : k) | (k > 1 ? k << 32 : 0);
}
// Part `number` of all, or (INNER) of those that are not the last of their
// sequence: whole ones, at most rows / part.  Found by a whole warp: lanes take
// 32 sequences at a time and scan their counts (which stay below 2^32: the host
// limits rows to 2^31 with cu).
template <bool INNER>
__device__ __forceinline__ Part find_part(const Seqs& q, int64_t part, int64_t number) {
  Part r;
  if (!q.cu) {
    const int64_t per = parts_of(q.each, part), each = INNER ? per - 1 : per;
    if (each == 0) return r;
    const int64_t s =
        static_cast<uint32_t>(number) / static_cast<uint32_t>(each);  // (a grid's index)
    if (s >= q.seqs) return r;
    r.seq = s;
    r.index = number - s * each;
    r.count = per;
    r.place = s * per + r.index;
    r.begin = s * q.each + r.index * part;
    const int64_t e = (s + 1) * q.each;
    r.end = r.begin + part < e ? r.begin + part : e;
    return r;
  }
  const int lane = threadIdx.x & 31;
  uint64_t before = 0;
  for (int64_t base = 0; base < q.seqs; base += 32) {
    int64_t b = 0, e = 0;
    uint64_t n = 0;
    if (base + lane < q.seqs) {
      seq_range(q, base + lane, b, e);
      n = part_counts<INNER>(e - b, part);
    }
    uint64_t inc = n;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    inc += before;
    const unsigned m =
        __ballot_sync(0xffffffffu, number < static_cast<int64_t>(inc & 0xffffffffu));
    if (m) {
      const int l = __ffs(m) - 1;
      const uint64_t k = __shfl_sync(0xffffffffu, inc - n, l);  // counts before the sequence
      b = __shfl_sync(0xffffffffu, b, l);
      e = __shfl_sync(0xffffffffu, e, l);
      r.seq = base + l;
      r.index = number - static_cast<int64_t>(k & 0xffffffffu);
      r.count = parts_of(e - b, part);
      r.place = static_cast<int64_t>(k >> 32) + r.index;
      r.begin = b + r.index * part;
      r.end = r.begin + part < e ? r.begin + part : e;
      return r;
    }
    before = __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// ---------------------------------------------------------------------------
// Host checks.
// ---------------------------------------------------------------------------
namespace mixer {

inline int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }
inline bool aligned_to(const void* p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// A buffer's bytes: rows of `width` elements, `stride` apart.
struct Buffer {
  const void* p;
  int64_t bytes;
};
// False when the extent does not fit in int64 or a stride is below the width.
inline bool extent(const void* p, int64_t rows, int64_t width, int64_t stride, int es, Buffer* b) {
  b->p = p;
  b->bytes = 0;
  if (!p || rows <= 0) return true;
  if (rows > 1 && stride < width) return false;
  const __int128 n =
      (static_cast<__int128>(rows - 1) * (rows > 1 ? stride : 0) + width) * es;
  if (n > static_cast<__int128>(INT64_MAX)) return false;
  b->bytes = static_cast<int64_t>(n);
  return true;
}
inline bool overlap(const Buffer& a, const Buffer& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// The same of two matrices of more than one row with one row stride (bytes): columns
// beside each other in the same rows do not overlap.
struct Columns {
  Buffer b;
  int64_t width, stride;  // bytes; stride 0: not rows that can interleave
};
inline Columns columns(const Buffer& b, int64_t rows, int64_t width, int64_t stride, int es) {
  return {b, width * es, rows > 1 ? stride * es : 0};
}
inline bool overlap(const Columns& a, const Columns& b) {
  if (!overlap(a.b, b.b)) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.b.p) -
                                   reinterpret_cast<uintptr_t>(a.b.p)) % a.stride;
  if (d < 0) d += a.stride;
  return !(d >= a.width && d <= a.stride - b.width);
}
// Whether an output overlaps another buffer: an input, or another output.
inline bool outputs_overlap(std::initializer_list<Columns> outs,
                            std::initializer_list<Columns> ins) {
  for (const Columns& o : outs) {
    for (const Columns& i : ins)
      if (overlap(o, i)) return true;
    for (const Columns& i : outs)
      if (&i != &o && overlap(o, i)) return true;
  }
  return false;
}

// Whether `rows` rows can be `seqs` sequences (of equal length without offsets).
inline bool counts_ok(int64_t rows, int64_t seqs, bool offsets) {
  if (rows < 0 || seqs < 0 || (seqs == 0 && rows > 0)) return false;
  if (!offsets && seqs > 0 && rows % seqs != 0) return false;
  return rows <= INT64_MAX / 2 && seqs <= INT32_MAX && !(offsets && rows > INT32_MAX);
}

// Checks of rows, sequences and the pool shared by every entry point.
// `step`: one row a sequence, the state required.
inline int check_seqs(int64_t rows, int64_t seqs, const int32_t* cu, const void* state,
                      const int32_t* slots, const uint8_t* resume, int64_t state_slots,
                      int64_t slot_width, int64_t slot_stride, bool step, Seqs* q) {
  if (step) {
    seqs = rows;
    cu = nullptr;
    resume = nullptr;
  }
  if (!counts_ok(rows, seqs, cu != nullptr)) return GGRN_ERR_SHAPE;
  if (!aligned_to(cu, 4) || !aligned_to(slots, 4)) return GGRN_ERR_ALIGN;
  if (!state) {
    if (step && rows > 0) return GGRN_ERR_NULL;
    if (slots || resume) return GGRN_ERR_ARG;
    state_slots = 0;
  } else {
    if (state_slots < 0 || (state_slots > 1 && slot_stride < slot_width)) return GGRN_ERR_SHAPE;
    if (!slots && state_slots < seqs) return GGRN_ERR_SHAPE;
  }
  q->cu = cu;
  q->slots = slots;
  q->resume = resume;
  q->rows = rows;
  q->seqs = seqs;
  q->each = cu || seqs == 0 ? 0 : rows / seqs;
  q->state_slots = state_slots;
  return GGRN_OK;
}

// Launch with programmatic dependent launch allowed (every kernel waits for
// its predecessor before it touches global memory).
template <typename... P, typename... A>
int launch(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
           A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return GGRN_ERR_CUDA;
  }
  return GGRN_OK;
}

}  // namespace mixer

// SM count of the current device (152 without one).
int device_sms();

// The step forms for decode graphs: the argument checks alone, and the call.
int check_conv(const ggrn_conv_call& c, bool step);
int check_scan(const ggrn_scan_call& c, bool step);
int check_recur(const ggrn_recur_call& c, bool step);
int check_layer_norm(const ggrn_layer_norm_call& c);

}  // namespace ggrn
