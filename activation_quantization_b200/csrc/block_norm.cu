// Norms before and after a block, fused with the block's gate and residual:
//   u     = N_post(y) * act(gate)
//   r_out = residual_scale * r + branch_scale * u
//   h     = N_pre(r_out)
// (wush_norm is the last line alone, with h = N_pre(x)).
//
// The work is bound by memory: y, r and the gate are read once, r_out and h are
// written once, and about 20 operations an element lie between.  So a row stays in
// the registers of the threads that read it: each thread holds NV groups of eight
// consecutive elements, the statistics are block reductions over those registers
// (the variance of a layer norm is summed around the mean, in a second reduction),
// and no element is read again.
#include "rowops.cuh"

namespace wush {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxVec = 4;                                 // groups of eight elements a thread holds
constexpr int kMaxWidth = kMaxThreads * kMaxVec * 8;       // 32768
constexpr int kMinThreads = 128;                           // narrow rows share a CTA of this many threads

struct NormArgs {
  int kind, dt;
  const void* w;
  const void* b;
  float offset, eps;
};

struct Args {
  const void* y;
  const void* r;
  const void* gate;
  void* r_out;
  void* h;
  int64_t y_stride, r_stride, gate_stride, r_out_stride, h_stride;
  int y_dt, r_dt, gate_dt, h_dt, act;
  float residual_scale, branch_scale;
  NormArgs post, pre;
  int64_t rows;
  int d, row_threads;                                      // threads of one row (a multiple of 32)
};

// Sum over the row's threads, the same in all of them and independent of timing: a
// shuffle tree in each warp, then the warps' sums in their order.
__device__ __forceinline__ float row_sum(float s, float* red, int warps, int warp0) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (warps == 1) return s;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0f;
  for (int i = 0; i < warps; ++i) s += red[warp0 + i];
  return s;
}

__device__ __forceinline__ float activate(float g, int act) {
  if (act == WUSH_GATE_LINEAR) return g;
  const float s = 1.0f / (1.0f + expf(-g));
  return act == WUSH_GATE_SIGMOID ? s : g * s;
}

// VEC: every pointer and stride is a multiple of 16 bytes and d of 8, so a thread's
// eight elements are one or two 16-byte accesses.  Otherwise the eight elements lie
// row_threads apart, so that a warp's single-element accesses are contiguous.
template <bool VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_kernel(const __grid_constant__ Args a) {
  __shared__ float red[4][32];
  const int g = a.row_threads, warps = g >> 5;
  const int sub = threadIdx.x / g, tid = threadIdx.x - sub * g, warp0 = sub * warps;
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / g) + sub;
  const bool live = row < a.rows;                          // the others only take part in the barriers
  const int d = live ? a.d : 0;
  float v[NV][8];

  auto column = [&](int j, int e) { return VEC ? (j * g + tid) * 8 + e : (j * 8 + e) * g + tid; };
  auto load = [&](const void* p, int dt, int64_t base, int j, float (&x)[8]) {
    if (VEC) {
      if (column(j, 0) < d) load8(p, dt, base + column(j, 0), x);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = column(j, e) < d ? load1(p, dt, base + column(j, e)) : 0.0f;
    }
  };
  auto store = [&](void* p, int dt, int64_t base, int j, const float (&x)[8]) {
    if (VEC) {
      if (column(j, 0) < d) store8(p, dt, base + column(j, 0), x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (column(j, e) < d) store1(p, dt, base + column(j, e), x[e]);
    }
  };
  auto norm = [&](const NormArgs& n, int phase) {
    if (n.kind == WUSH_ROWNORM_NONE) return;
    float s = 0.0f;
    if (n.kind == WUSH_ROWNORM_LAYER) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[j][e];
      const float mean = row_sum(s, red[phase], warps, warp0) / static_cast<float>(a.d);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = column(j, e) < d ? v[j][e] - mean : 0.0f;
      s = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
    const float f = 1.0f / sqrtf(row_sum(s, red[phase + 1], warps, warp0) / static_cast<float>(a.d) + n.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (n.w) {
        float w[8];
        load(n.w, n.dt, 0, j, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * f * (w[e] + n.offset);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= f;
      }
      if (n.b) {
        float b[8];
        load(n.b, n.dt, 0, j, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] += b[e];
      }
    }
  };

  const int64_t r_base = row * a.r_stride;
  if (a.y) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load(a.y, a.y_dt, row * a.y_stride, j, v[j]);
    norm(a.post, 0);
    if (a.gate) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load(a.gate, a.gate_dt, row * a.gate_stride, j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= activate(x[e], a.act);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      if (a.r) {
        load(a.r, a.r_dt, r_base, j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = fmaf(a.branch_scale, v[j][e], a.residual_scale * x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= a.branch_scale;
      }
      if (a.r_out) store(a.r_out, a.r_dt, row * a.r_out_stride, j, v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) load(a.r, a.r_dt, r_base, j, v[j]);
  }
  if (a.h) {
    norm(a.pre, 2);
#pragma unroll
    for (int j = 0; j < NV; ++j) store(a.h, a.h_dt, row * a.h_stride, j, v[j]);
  }
}

// ------------------------------------------------------------------ host checks

bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_norm(const wush_norm_spec* s, NormArgs* out, bool* vec) {
  *out = NormArgs{WUSH_ROWNORM_NONE, WUSH_FP32, nullptr, nullptr, 0.0f, 0.0f};
  if (s->kind == WUSH_ROWNORM_NONE) return WUSH_OK;
  if (s->kind != WUSH_ROWNORM_RMS && s->kind != WUSH_ROWNORM_LAYER) return WUSH_ERR_UNSUPPORTED;
  if (!(s->eps >= 0.0f) || !(s->eps < 3.0e38f)) return WUSH_ERR_INVALID_ARG;
  if (!(s->weight_offset > -3.0e38f && s->weight_offset < 3.0e38f)) return WUSH_ERR_INVALID_ARG;
  if (s->weight || s->bias) {
    if (!known_dtype(s->dtype)) return WUSH_ERR_UNSUPPORTED;
    for (const void* p : {s->weight, s->bias}) {
      if (!aligned_to(p, dtype_bytes(s->dtype))) return WUSH_ERR_INVALID_ARG;
      *vec = *vec && aligned_to(p, 16);
    }
  }
  *out = NormArgs{s->kind, s->dtype, s->weight, s->bias, s->weight_offset, s->eps};
  return WUSH_OK;
}

// One tensor's rows: its type, alignment and stride (0 only where ``broadcast``).
int check_rows(const void* p, int dt, int64_t stride, int64_t rows, int64_t d, bool broadcast, bool* vec) {
  if (!p) return WUSH_OK;
  if (!known_dtype(dt)) return WUSH_ERR_UNSUPPORTED;
  if (!aligned_to(p, dtype_bytes(dt))) return WUSH_ERR_INVALID_ARG;
  if (!(broadcast && stride == 0) && stride < d) return WUSH_ERR_INVALID_ARG;
  if (stride > (int64_t(1) << 60) / (rows > 0 ? rows : 1)) return WUSH_ERR_UNSUPPORTED;
  *vec = *vec && aligned_to(p, 16) && stride * dtype_bytes(dt) % 16 == 0;
  return WUSH_OK;
}

template <bool VEC, int NV>
int launch(const Args& a, int block, cudaStream_t st) {
  const int64_t per = block / a.row_threads, grid = (a.rows + per - 1) / per;
  residual_norm_kernel<VEC, NV><<<static_cast<unsigned>(grid), block, 0, st>>>(a);
  return launch_status();
}

int run(Args& a, bool vec, cudaStream_t st) {
  const int groups = (a.d + 7) / 8;
  // Few rows: one group of eight a thread, so that a row's latency is one load deep.
  // Many rows: as many as fit, so that fewer threads meet in the reductions.
  int nv = 1;
  if (a.rows > 296) nv = groups >= 512 ? 4 : groups >= 128 ? 2 : 1;
  while (nv < kMaxVec && (groups + nv - 1) / nv > kMaxThreads) nv *= 2;
  int threads = (((groups + nv - 1) / nv) + 31) / 32 * 32;
  if (threads < kMinThreads) threads = threads <= 32 ? 32 : threads <= 64 ? 64 : kMinThreads;
  a.row_threads = threads;
  const int block = threads < kMinThreads ? kMinThreads : threads;
  if (vec) return nv == 1 ? launch<true, 1>(a, block, st) : nv == 2 ? launch<true, 2>(a, block, st) : launch<true, 4>(a, block, st);
  return nv == 1 ? launch<false, 1>(a, block, st) : nv == 2 ? launch<false, 2>(a, block, st) : launch<false, 4>(a, block, st);
}

}  // namespace
}  // namespace wush

using namespace wush;

extern "C" int wush_residual_norm(const wush_residual_norm_args* args, void* stream) {
  if (!args) return WUSH_ERR_INVALID_ARG;
  const wush_residual_norm_args& q = *args;
  const int64_t rows = q.rows, d = q.d;
  if (rows < 0 || d <= 0 || !q.y || (!q.r_out && !q.h)) return WUSH_ERR_INVALID_ARG;
  if (d > kMaxWidth || rows > 0x7fffffff) return WUSH_ERR_UNSUPPORTED;
  if (q.gate && (q.gate_act < WUSH_GATE_LINEAR || q.gate_act > WUSH_GATE_SILU)) return WUSH_ERR_UNSUPPORTED;
  if (!(q.residual_scale - q.residual_scale == 0.0f) || !(q.branch_scale - q.branch_scale == 0.0f))
    return WUSH_ERR_INVALID_ARG;
  bool vec = d % 8 == 0;
  Args a = {};
  int st;
  if ((st = check_rows(q.y, q.y_dtype, q.y_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_rows(q.gate, q.gate_dtype, q.gate_stride, rows, d, true, &vec)) != WUSH_OK) return st;
  if ((st = check_rows(q.r, q.r_dtype, q.r_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_rows(q.r_out, q.r_dtype, q.r_out_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_rows(q.h, q.h_dtype, q.h_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_norm(&q.post, &a.post, &vec)) != WUSH_OK) return st;
  if ((st = check_norm(&q.pre, &a.pre, &vec)) != WUSH_OK) return st;
  if (rows == 0) return WUSH_OK;
  const Span sy = span(q.y, q.y_dtype, q.y_stride, d), sr = span(q.r, q.r_dtype, q.r_stride, d),
             so = span(q.r_out, q.r_dtype, q.r_out_stride, d), sh = span(q.h, q.h_dtype, q.h_stride, d);
  const bool in_place = q.r_out && q.r_out == q.r && q.r_out_stride == q.r_stride;
  if (overlap(so, sy, rows) || (!in_place && overlap(so, sr, rows)) || overlap(sh, sy, rows) ||
      overlap(sh, sr, rows) || overlap(sh, so, rows))
    return WUSH_ERR_INVALID_ARG;
  for (const Span& out : {so, sh}) {
    if (!q.gate || !out.p) continue;
    const char* g = static_cast<const char*>(q.gate);
    // (a gate per channel is one row, read by every row)
    if (q.gate_stride ? overlap(out, span(q.gate, q.gate_dtype, q.gate_stride, d), rows)
                      : out.p < g + d * dtype_bytes(q.gate_dtype) && g < out.p + (rows - 1) * out.stride + out.width)
      return WUSH_ERR_INVALID_ARG;
  }
  a.y = q.y; a.y_dt = q.y_dtype; a.y_stride = q.y_stride;
  a.gate = q.gate; a.gate_dt = q.gate_dtype; a.gate_stride = q.gate_stride; a.act = q.gate_act;
  a.r = q.r; a.r_dt = q.r_dtype; a.r_stride = q.r_stride;
  a.r_out = q.r_out; a.r_out_stride = q.r_out_stride;
  a.h = q.h; a.h_dt = q.h_dtype; a.h_stride = q.h_stride;
  a.residual_scale = q.residual_scale; a.branch_scale = q.branch_scale;
  a.rows = rows; a.d = static_cast<int>(d);
  return run(a, vec, static_cast<cudaStream_t>(stream));
}

extern "C" int wush_norm(const void* x, int x_dtype, int64_t x_stride, int64_t rows, int64_t d,
                         const wush_norm_spec* norm, void* h, int h_dtype, int64_t h_stride, void* stream) {
  if (rows < 0 || d <= 0 || !x || !h || !norm) return WUSH_ERR_INVALID_ARG;
  if (d > kMaxWidth || rows > 0x7fffffff) return WUSH_ERR_UNSUPPORTED;
  bool vec = d % 8 == 0;
  Args a = {};
  int st;
  if ((st = check_rows(x, x_dtype, x_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_rows(h, h_dtype, h_stride, rows, d, false, &vec)) != WUSH_OK) return st;
  if ((st = check_norm(norm, &a.pre, &vec)) != WUSH_OK) return st;
  if (rows == 0) return WUSH_OK;
  const bool in_place = x == h && x_dtype == h_dtype && x_stride == h_stride;
  if (!in_place && overlap(span(h, h_dtype, h_stride, d), span(x, x_dtype, x_stride, d), rows))
    return WUSH_ERR_INVALID_ARG;
  a.r = x; a.r_dt = x_dtype; a.r_stride = x_stride;
  a.h = h; a.h_dt = h_dtype; a.h_stride = h_stride;
  a.rows = rows; a.d = static_cast<int>(d);
  return run(a, vec, static_cast<cudaStream_t>(stream));
}
