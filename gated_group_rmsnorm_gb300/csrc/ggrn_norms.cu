// ggrn_norms.cu -- layer norm and the backward passes of the norms: checks,
// layout and launches of the kernels in ggrn_norms.cuh, and the sum of what
// their CTAs leave of the weights' gradients.
#include <initializer_list>

#include "ggrn_norms.cuh"

namespace ggrn {
namespace norms {

// out[c] = the sum of in[k, c] over k < n, in a fixed order: 32 threads to a
// column, each every 32nd row.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) k_column_sum(const float* in0, const float* in1,
                                                              float* out0, float* out1, int64_t n,
                                                              int64_t columns) {
  __shared__ float s[kSumRows][32];
  pdl_wait();
  pdl_launch_dependents();
  const float* in = blockIdx.y ? in1 : in0;
  float* out = blockIdx.y ? out1 : out0;
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float t = 0.0f;
  if (c < columns) {
    // (eight reads in flight)
    for (int64_t k0 = row; k0 < n; k0 += 8 * kSumRows) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t k = k0 + i * kSumRows;
        v[i] = k < n ? in[k * columns + c] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[i];
    }
  }
  s[row][lane] = t;
  __syncthreads();
  if (row != 0 || c >= columns) return;
  for (int k = 1; k < kSumRows; ++k) t += s[k][lane];
  out[c] = t;
}

Plan plan(int kind, int es, int64_t rows, int64_t groups, int64_t gs, int elems) {
  Plan k;
  k.elems = elems;
  const int64_t nvec = gs / elems;
  int vpl = team_elems(kind) / elems;
  vpl = vpl > 4 ? 4 : vpl;
  int lanes = 1;
  while (lanes < 32 && lanes * vpl < nvec) lanes <<= 1;
  if (nvec <= lanes * vpl) {
    // several groups to a CTA
    k.vpl = nvec <= lanes ? 1 : nvec <= 2 * lanes ? 2 : 4;
    k.lanes = lanes;
    const int teams = 256 / lanes;
    const int64_t blocks = (groups + teams - 1) / teams;  // as full as each other
    k.team_groups = static_cast<int>((groups + blocks - 1) / blocks);
    k.team_rows = teams / k.team_groups;
    k.threads = (k.team_groups * k.team_rows * lanes + 31) / 32 * 32;
  } else {
    // a CTA to a group.  Layer norm: as many vectors a thread as it holds well (16384
    // rows of 3840: 46 us with four, 64 with one, whose sums take more threads).  The
    // gradients: those that give an SM the most threads, the more of two alike.
    k.vpl = 0;
    int64_t most = 0;
    for (int v = 1; v <= 4; v *= 2) {
      const int64_t threads = ((nvec + v - 1) / v + 31) / 32 * 32;
      if (threads > threads_of(kind, v * elems) ||
          threads * v * elems * es * inputs_of(kind) * depth_of(kind) > kRingMost)
        continue;
      const int64_t held = room_of(kind, v * elems) / threads * threads;
      if (k.vpl && (v * elems > cta_elems(kind) || (kind != kLayerNorm && held < most))) continue;
      most = held;
      k.vpl = v;
      k.threads = static_cast<int>(threads);
    }
    if (k.vpl == 0) k.threads = kAnyThreads;
    k.lanes = k.threads;
  }
  k.nvec = static_cast<int>(k.vpl ? nvec : 0);
  k.blocks = (groups + k.team_groups - 1) / k.team_groups;
  const int64_t sms = device_sms();
  int64_t resident = 2048 / k.threads;
  if (k.vpl) {
    resident = room_of(kind, k.vpl * elems) / k.threads;
    const int row = inputs_of(kind) * k.vpl * k.threads * elems * es;
    const int most = (220 << 10) / (depth_of(kind) * row + 2048);
    if (resident > most) resident = most;
    if (resident > 16) resident = 16;
    if (resident < 1) resident = 1;
    k.smem = depth_of(kind) * row;
  }
  // (gradients: a CTA's sums are a row for k_column_sum to read, so a CTA takes at
  // least two rows of a group: 300 rows of 4800 11.0 us, with one 13.0, with four 12.5)
  const int64_t turn = k.team_rows * (kind == kLayerNorm ? 1 : 2);
  const int64_t most = (rows + turn - 1) / turn;
  k.slices = (sms * resident) / k.blocks;
  if (k.slices > most) k.slices = most;
  if (k.slices < 1) k.slices = 1;
  if (kind != kLayerNorm) {
    k.sums = kind == kOnnxGrad ? k.slices * k.blocks : k.slices;
    k.columns = kind == kOnnxGrad ? gs : groups * gs;
    const int acc = k.threads * k.elems * k.vpl * 4;  // (the ring's place, at the end)
    if (k.smem < acc) k.smem = acc;
  }
  return k;
}

// Elements of a vector that every row of every matrix can be read by: 16 bytes,
// 8 bytes, or one.
struct Matrix {
  const void* p;
  int64_t stride;
};
int elements(int es, int64_t rows, int64_t gs, std::initializer_list<Matrix> ms) {
  for (int bytes : {16, 8}) {
    bool fits = gs * es % bytes == 0;
    for (const Matrix& m : ms)
      fits = fits && mixer::aligned_to(m.p, bytes) && (rows <= 1 || m.stride * es % bytes == 0);
    if (fits) return bytes / es;
  }
  return 1;
}

// Bytes of the partial sums, whatever the alignment of the call's matrices.
int64_t space(int kind, int es, int64_t rows, int64_t groups, int64_t gs) {
  int64_t most = 0;
  if (rows == 0) return 0;
  for (int elems : {16 / es, 8 / es, 1}) {
    if (gs % elems) continue;
    const Plan k = plan(kind, es, rows, groups, gs, elems);
    if (k.sums <= 1) continue;
    const int64_t bytes = k.sums * k.columns * 4 * (kind == kLayerNormGrad ? 2 : 1);
    if (bytes > most) most = bytes;
  }
  return most;
}

// Sizes that a group's columns and a grid can have.
int check_sizes(int dtype, int64_t rows, int64_t width, int64_t gs) {
  if (dtype != kF32 && dtype != kF16 && dtype != kBF16) return GGRN_ERR_DTYPE;
  if (rows < 0 || width <= 0 || gs <= 0 || width % gs != 0) return GGRN_ERR_SHAPE;
  if (width > int64_t{1} << 40 || rows > INT64_MAX / 2) return GGRN_ERR_SHAPE;
  // (a group of more than 32 elements may take a CTA of its own)
  if (width / gs > 65535 * (gs <= 32 ? int64_t{8} : 1)) return GGRN_ERR_UNSUPPORTED;
  return GGRN_OK;
}

int launch(int kind, int dtype, Params& p, const Plan& k, void* workspace, float* dw, float* db,
           cudaStream_t s) {
  p.lanes = k.lanes;
  p.team_groups = k.team_groups;
  p.team_rows = k.team_rows;
  p.nvec = k.nvec;
  p.gs_f = static_cast<float>(p.gs);
  p.inv_gs = 1.0f / static_cast<float>(p.gs);
  float* const sums = static_cast<float*>(workspace);
  p.dw = k.sums > 1 ? sums : dw;
  p.db = !db ? nullptr : k.sums > 1 ? sums + k.sums * k.columns : db;
  const int st = dtype == kF32   ? launch_f32(kind, p, k, s)
                 : dtype == kF16 ? launch_f16(kind, p, k, s)
                                 : launch_bf16(kind, p, k, s);
  if (st != GGRN_OK || k.sums <= 1) return st;
  return mixer::launch(k_column_sum,
                       dim3(static_cast<unsigned>((k.columns + 31) / 32), db ? 2 : 1),
                       32 * kSumRows, 0, s, static_cast<const float*>(p.dw),
                       static_cast<const float*>(p.db), dw, db, k.sums, k.columns);
}
int launch_zeros(float* dw, float* db, int64_t columns, cudaStream_t s) {
  return mixer::launch(k_column_sum, dim3(static_cast<unsigned>((columns + 31) / 32), db ? 2 : 1),
                       32 * kSumRows, 0, s, static_cast<const float*>(nullptr),
                       static_cast<const float*>(nullptr), dw, db, int64_t{0}, columns);
}

// A matrix of the call, and a vector of n bytes.
mixer::Columns matrix(const mixer::Buffer& b, int64_t rows, int64_t width, int64_t stride, int es) {
  return mixer::columns(b, rows, width, stride, es);
}
mixer::Columns vector(const void* p, int64_t n) { return {{p, n}, 0, 0}; }

int check_layer_norm(const ggrn_layer_norm_call& c) {
  const int st = check_sizes(c.dtype, c.rows, c.width, c.width);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  mixer::Buffer x, out;
  if (!mixer::extent(c.x, c.rows, c.width, c.x_row_stride, es, &x) ||
      !mixer::extent(c.out, c.rows, c.width, c.out_row_stride, es, &out))
    return GGRN_ERR_SHAPE;
  if (c.rows == 0) return GGRN_OK;
  if (!c.x || !c.w || !c.out) return GGRN_ERR_NULL;
  if (!mixer::aligned_to(c.x, es) || !mixer::aligned_to(c.out, es) || !mixer::aligned_to(c.w, 4) ||
      !mixer::aligned_to(c.b, 4))
    return GGRN_ERR_ALIGN;
  return mixer::outputs_overlap({matrix(out, c.rows, c.width, c.out_row_stride, es)},
                                {matrix(x, c.rows, c.width, c.x_row_stride, es),
                                 vector(c.w, c.width * 4), vector(c.b, c.width * 4)})
             ? GGRN_ERR_OVERLAP
             : GGRN_OK;
}

int run(const ggrn_layer_norm_call* call, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_layer_norm_call& c = *call;
  const int st = check_layer_norm(c);
  if (st != GGRN_OK || c.rows == 0) return st;
  const int es = mixer::elem_bytes(c.dtype);
  Params p = {};
  p.x = c.x;
  p.w = c.w;
  p.b = c.b;
  p.out = c.out;
  p.rows = c.rows;
  p.groups = 1;
  p.gs = c.width;
  p.xs = c.rows > 1 ? c.x_row_stride : 0;
  p.os = c.rows > 1 ? c.out_row_stride : 0;
  p.eps = c.eps;
  const Plan k = plan(kLayerNorm, es, c.rows, 1, c.width,
                      elements(es, c.rows, c.width, {{c.x, p.xs}, {c.out, p.os}}));
  return launch(kLayerNorm, c.dtype, p, k, nullptr, nullptr, nullptr,
                static_cast<cudaStream_t>(stream));
}

int run(const ggrn_layer_norm_backward_call* call, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_layer_norm_backward_call& c = *call;
  const int st = check_sizes(c.dtype, c.rows, c.width, c.width);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  mixer::Buffer x, dout, dx;
  if (!mixer::extent(c.x, c.rows, c.width, c.x_row_stride, es, &x) ||
      !mixer::extent(c.dout, c.rows, c.width, c.dout_row_stride, es, &dout) ||
      !mixer::extent(c.dx, c.rows, c.width, c.dx_row_stride, es, &dx))
    return GGRN_ERR_SHAPE;
  if (!c.dw || (c.rows > 0 && (!c.x || !c.dout || !c.dx || !c.w))) return GGRN_ERR_NULL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t need = space(kLayerNormGrad, es, c.rows, 1, c.width);
  if (need > 0 && !c.workspace) return GGRN_ERR_NULL;
  if (!mixer::aligned_to(c.x, es) || !mixer::aligned_to(c.dout, es) ||
      !mixer::aligned_to(c.dx, es) || !mixer::aligned_to(c.w, 4) || !mixer::aligned_to(c.dw, 4) ||
      !mixer::aligned_to(c.db, 4) || (need > 0 && !mixer::aligned_to(c.workspace, 16)))
    return GGRN_ERR_ALIGN;
  if (need > 0 && c.workspace_bytes < need) return GGRN_ERR_ARG;
  if (mixer::outputs_overlap({matrix(dx, c.rows, c.width, c.dx_row_stride, es),
                              vector(c.dw, c.width * 4), vector(c.db, c.width * 4),
                              vector(c.workspace, need)},
                             {matrix(x, c.rows, c.width, c.x_row_stride, es),
                              matrix(dout, c.rows, c.width, c.dout_row_stride, es),
                              vector(c.w, c.width * 4)}))
    return GGRN_ERR_OVERLAP;
  if (c.rows == 0) return launch_zeros(c.dw, c.db, c.width, s);
  Params p = {};
  p.x = c.x;
  p.dout = c.dout;
  p.w = c.w;
  p.out = c.dx;
  p.rows = c.rows;
  p.groups = 1;
  p.gs = c.width;
  p.xs = c.rows > 1 ? c.x_row_stride : 0;
  p.ds = c.rows > 1 ? c.dout_row_stride : 0;
  p.os = c.rows > 1 ? c.dx_row_stride : 0;
  p.eps = c.eps;
  const Plan k = plan(kLayerNormGrad, es, c.rows, 1, c.width,
                      elements(es, c.rows, c.width, {{c.x, p.xs}, {c.dout, p.ds}, {c.dx, p.os}}));
  return launch(kLayerNormGrad, c.dtype, p, k, c.workspace, c.dw, c.db, s);
}

int run(const ggrn_backward_call* call, void* stream) {
  if (!call) return GGRN_ERR_ARG;
  const ggrn_backward_call& c = *call;
  if (c.mode != kMamba2 && c.mode != kOnnx) return GGRN_ERR_DTYPE;
  if (c.mode == kOnnx && c.dtype == kBF16) return GGRN_ERR_DTYPE;
  const int st = check_sizes(c.dtype, c.rows, c.width, c.group_size);
  if (st != GGRN_OK) return st;
  const int es = mixer::elem_bytes(c.dtype);
  mixer::Buffer dout, y, gate, dy, dgate;
  if (!mixer::extent(c.dout, c.rows, c.width, c.dout_row_stride, es, &dout) ||
      !mixer::extent(c.y, c.rows, c.width, c.y_row_stride, es, &y) ||
      !mixer::extent(c.gate, c.rows, c.width, c.gate_row_stride, es, &gate) ||
      !mixer::extent(c.dy, c.rows, c.width, c.dy_row_stride, es, &dy) ||
      !mixer::extent(c.dgate, c.rows, c.width, c.dgate_row_stride, es, &dgate))
    return GGRN_ERR_SHAPE;
  if (!c.dw || (c.rows > 0 && (!c.dout || !c.y || !c.gate || !c.w || !c.dy || !c.dgate)))
    return GGRN_ERR_NULL;
  const int kind = c.mode == kOnnx ? kOnnxGrad : kMamba2Grad, wes = c.mode == kOnnx ? es : 4;
  const int64_t groups = c.width / c.group_size, columns = c.mode == kOnnx ? c.group_size : c.width;
  const int64_t need = space(kind, es, c.rows, groups, c.group_size);
  if (need > 0 && !c.workspace) return GGRN_ERR_NULL;
  for (const void* q : {c.dout, c.y, c.gate, static_cast<const void*>(c.dy),
                        static_cast<const void*>(c.dgate)})
    if (!mixer::aligned_to(q, es)) return GGRN_ERR_ALIGN;
  if (!mixer::aligned_to(c.w, wes) || !mixer::aligned_to(c.dw, 4) ||
      (need > 0 && !mixer::aligned_to(c.workspace, 16)))
    return GGRN_ERR_ALIGN;
  if (need > 0 && c.workspace_bytes < need) return GGRN_ERR_ARG;
  if (mixer::outputs_overlap({matrix(dy, c.rows, c.width, c.dy_row_stride, es),
                              matrix(dgate, c.rows, c.width, c.dgate_row_stride, es),
                              vector(c.dw, columns * 4), vector(c.workspace, need)},
                             {matrix(dout, c.rows, c.width, c.dout_row_stride, es),
                              matrix(y, c.rows, c.width, c.y_row_stride, es),
                              matrix(gate, c.rows, c.width, c.gate_row_stride, es),
                              vector(c.w, columns * wes)}))
    return GGRN_ERR_OVERLAP;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c.rows == 0) return launch_zeros(c.dw, nullptr, columns, s);
  Params p = {};
  p.dout = c.dout;
  p.x = c.y;
  p.gate = c.gate;
  p.w = c.w;
  p.out = c.dy;
  p.dgate = c.dgate;
  p.rows = c.rows;
  p.groups = groups;
  p.gs = c.group_size;
  const bool many = c.rows > 1;
  p.ds = many ? c.dout_row_stride : 0;
  p.xs = many ? c.y_row_stride : 0;
  p.gts = many ? c.gate_row_stride : 0;
  p.os = many ? c.dy_row_stride : 0;
  p.dgs = many ? c.dgate_row_stride : 0;
  p.eps = c.eps;
  const Plan k = plan(kind, es, c.rows, groups, c.group_size,
                      elements(es, c.rows, c.group_size,
                               {{c.dout, p.ds}, {c.y, p.xs}, {c.gate, p.gts}, {c.dy, p.os},
                                {c.dgate, p.dgs}}));
  return launch(kind, c.dtype, p, k, c.workspace, c.dw, nullptr, s);
}

}  // namespace norms

int check_layer_norm(const ggrn_layer_norm_call& c) { return norms::check_layer_norm(c); }

}  // namespace ggrn

extern "C" int ggrn_layer_norm(const ggrn_layer_norm_call* call, void* cuda_stream) {
  return ggrn::norms::run(call, cuda_stream);
}
extern "C" int ggrn_layer_norm_backward(const ggrn_layer_norm_backward_call* call,
                                        void* cuda_stream) {
  return ggrn::norms::run(call, cuda_stream);
}
extern "C" int ggrn_backward(const ggrn_backward_call* call, void* cuda_stream) {
  return ggrn::norms::run(call, cuda_stream);
}
extern "C" int64_t ggrn_layer_norm_backward_workspace_bytes(
    const ggrn_layer_norm_backward_call* c) {
  using namespace ggrn;
  if (!c || norms::check_sizes(c->dtype, c->rows, c->width, c->width) != GGRN_OK) return 0;
  return norms::space(norms::kLayerNormGrad, mixer::elem_bytes(c->dtype), c->rows, 1, c->width);
}
extern "C" int64_t ggrn_backward_workspace_bytes(const ggrn_backward_call* c) {
  using namespace ggrn;
  if (!c || (c->mode != kMamba2 && c->mode != kOnnx) ||
      norms::check_sizes(c->dtype, c->rows, c->width, c->group_size) != GGRN_OK)
    return 0;
  return norms::space(c->mode == kOnnx ? norms::kOnnxGrad : norms::kMamba2Grad,
                      mixer::elem_bytes(c->dtype), c->rows, c->width / c->group_size,
                      c->group_size);
}
