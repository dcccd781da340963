// Norms before and after a block, fused with the block's gate and residual:
//   u     = N_post(y) * act(gate)
//   r_out = residual_scale * r + branch_scale * u
//   h     = N_pre(r_out)
// (wush_norm is the last line alone, with h = N_pre(x)).
//
// The work is bound by memory: y, r and the gate are read once, r_out and h are
// written once, and about 20 operations an element lie between.  A row is held in the
// registers of the threads that work on it; the statistics are block reductions over
// those registers (a layer norm's variance is summed around the mean, in a second
// reduction), and no element is read from memory twice.
//
// Two kernels share that arithmetic:
//  * few rows: one CTA a row, loads straight to registers (latency counts);
//  * many rows: persistent CTAs, each with a ring of whole rows in shared memory that
//    bulk copies fill ahead of it, so that the bytes in flight do not depend on how
//    many threads wait.
#include "rowops.cuh"
#include "sm100.cuh"

namespace wush {

static __device__ int g_norm_error = 0;

int read_and_clear_norm_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_norm_error, sizeof(int));
  if (e != cudaSuccess) return e;
  if (*word) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(int));
  }
  return e;
}

namespace {

using sm100::mbar_init;

constexpr int kMaxWidth = 32768;
constexpr int kMaxStages = 4;
constexpr int kMinThreads = 128;                           // few rows: narrow ones share a CTA of this many threads
constexpr int64_t kDefaultPolls = int64_t(1) << 40;        // waits end on the timer
constexpr uint64_t kDeadlineNs = 4000000000ull;

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
  float inv_d;
};

// Where the ring kernel keeps things (bytes from the start of its shared memory; -1:
// not in shared memory, read where it lies).
struct Ring {
  int stages;
  int y, r, gate;                                          // first stage of each tensor's rows
  int y_step, r_step, gate_step;                           // from one stage to the next
  int vec[5];                                              // post w, post b, pre w, pre b, gate per channel
  bool kept;                                               // the vectors are in shared memory
};

__device__ __forceinline__ float activate(float g, int act) {
  if (act == WUSH_GATE_LINEAR) return g;
  const float s = 1.0f / (1.0f + expf(-g));
  return act == WUSH_GATE_SIGMOID ? s : g * s;
}

// Sum over the row's warps, the same in all of its threads and independent of timing: a
// shuffle tree in each warp, then the warps' sums in their order (``red``: 32 floats,
// zeros beyond the CTA's warps).
__device__ __forceinline__ float row_sum(float s, float* red, int warps, int warp0) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (warps == 1) return s;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0f;
  if (warps & 3) {
    for (int i = 0; i < warps; ++i) s += red[warp0 + i];
  } else {
    for (int i = 0; i < warps; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(red + warp0 + i);
      s += q.x; s += q.y; s += q.z; s += q.w;
    }
  }
  return s;
}

// v = N(v) over the row; ``w`` and ``b`` are the vectors, wherever they lie.
template <bool VEC, int NV>
__device__ __forceinline__ void apply_norm(const Args& a, const NormArgs& n, const void* w, const void* b,
                                           float (&v)[NV][8], float (*red)[32], int g, int tid, int warp0, int d) {
  if (n.kind == WUSH_ROWNORM_NONE) return;
  const int warps = g >> 5;
  float s = 0.0f;
  if (n.kind == WUSH_ROWNORM_LAYER) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[j][e];
    const float mean = row_sum(s, red[0], warps, warp0) * a.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = group_column<VEC>(j, e, g, tid) < d ? v[j][e] - mean : 0.0f;
    s = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
  const float f = rsqrtf(fmaf(row_sum(s, red[1], warps, warp0), a.inv_d, n.eps));
  if (w) {
    with_dtype(n.dt, [&](auto dt) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<dt.value, VEC>(w, j, g, tid, d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * f * (x[e] + n.offset);
      }
    });
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= f;
  }
  if (b) {
    with_dtype(n.dt, [&](auto dt) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<dt.value, VEC>(b, j, g, tid, d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] += x[e];
      }
    });
  }
}

template <bool VEC, int NV>
__device__ __forceinline__ void load_row(const void* row, int dt, int g, int tid, int d, float (&v)[NV][8]) {
  with_dtype(dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_group<t.value, VEC>(row, j, g, tid, d, v[j]);
  });
}

template <bool VEC, int NV>
__device__ __forceinline__ void store_row(void* row, int dt, int g, int tid, int d, const float (&v)[NV][8]) {
  with_dtype(dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) store_group<t.value, VEC>(row, j, g, tid, d, v[j]);
  });
}

// v = residual_scale * r + branch_scale * v * act(gate)
template <bool VEC, int NV>
__device__ __forceinline__ void gate_and_add(const Args& a, const void* gate, const void* r, float (&v)[NV][8], int g,
                                             int tid, int d) {
  if (gate)
    with_dtype(a.gate_dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<t.value, VEC>(gate, j, g, tid, d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= activate(x[e], a.act);
      }
    });
  if (r) {
    with_dtype(a.r_dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<t.value, VEC>(r, j, g, tid, d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = fmaf(a.branch_scale, v[j][e], a.residual_scale * x[e]);
      }
    });
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= a.branch_scale;
  }
}

// ---------------------------------------------------------------------------
// Few rows: one CTA a row (narrow rows share one).
// ---------------------------------------------------------------------------
template <bool VEC>
__global__ void __launch_bounds__(1024) norm_few_kernel(const __grid_constant__ Args a) {
  __shared__ __align__(16) float red[4][32];
  const int g = a.row_threads, sub = threadIdx.x / g, tid = threadIdx.x - sub * g, warp0 = sub * (g >> 5);
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / g) + sub;
  const bool live = row < a.rows;                          // the others only take part in the barriers
  const int d = live ? a.d : 0;
  float v[1][8];
  const void* r = a.r ? row_of(a.r, a.r_dt, row * a.r_stride) : nullptr;
  if (a.y) {
    load_row<VEC, 1>(row_of(a.y, a.y_dt, row * a.y_stride), a.y_dt, g, tid, d, v);
    apply_norm<VEC, 1>(a, a.post, a.post.w, a.post.b, v, red, g, tid, warp0, d);
    gate_and_add<VEC, 1>(a, a.gate ? row_of(a.gate, a.gate_dt, row * a.gate_stride) : nullptr, r, v, g, tid, d);
    if (a.r_out) store_row<VEC, 1>(row_of(a.r_out, a.r_dt, row * a.r_out_stride), a.r_dt, g, tid, d, v);
  } else {
    load_row<VEC, 1>(r, a.r_dt, g, tid, d, v);
  }
  if (a.h) {
    apply_norm<VEC, 1>(a, a.pre, a.pre.w, a.pre.b, v, red + 2, g, tid, warp0, d);
    store_row<VEC, 1>(row_of(a.h, a.h_dt, row * a.h_stride), a.h_dt, g, tid, d, v);
  }
}

// ---------------------------------------------------------------------------
// Many rows: a ring of rows in shared memory.
//
// A stage of a tensor holds one row at the 16-byte phase that the row has in global
// memory.  The whole 16-byte units of the row come by a bulk copy; what is left at its
// ends when rows are not aligned (VEC false) is copied by single threads.  y has a
// barrier of its own, r and the gate share one: y's stage is refilled as soon as the
// first reduction has read it, the others' after the second.
// ---------------------------------------------------------------------------
template <bool VEC, int NV, int G>
__global__ void __launch_bounds__(G, 1024 / G) norm_ring_kernel(const __grid_constant__ Args a,
                                                         const __grid_constant__ Ring q) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float red[2][4][32];
  __shared__ __align__(8) uint64_t full[2][kMaxStages];    // [y | r and gate]
  __shared__ int abort_flag;
  constexpr int g = G;                                     // (a constant, so that columns are immediate offsets)
  const int tid = threadIdx.x, d = a.d;
  const bool gate_rows = a.gate && a.gate_stride;
  const int64_t n_rows = blockIdx.x < a.rows ? (a.rows - 1 - blockIdx.x) / gridDim.x + 1 : 0;

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[0][i], 1);
      mbar_init(&full[1][i], 1);
    }
    sm100::fence_barrier_init();
  }
  for (int i = tid; i < 2 * 4 * 32; i += g) (&red[0][0][0])[i] = 0.0f;
  // the vectors that every row uses
  const void* vec[5] = {a.post.w, a.post.b, a.pre.w, a.pre.b, gate_rows ? nullptr : a.gate};
  const int vec_dt[5] = {a.post.dt, a.post.dt, a.pre.dt, a.pre.dt, a.gate_dt};
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (!vec[k] || q.vec[k] < 0) continue;
    if (vec_dt[k] == WUSH_FP32) {
      for (int i = tid; i < d; i += g)
        reinterpret_cast<uint32_t*>(smem + q.vec[k])[i] = static_cast<const uint32_t*>(vec[k])[i];
    } else {
      for (int i = tid; i < d; i += g)
        reinterpret_cast<uint16_t*>(smem + q.vec[k])[i] = static_cast<const uint16_t*>(vec[k])[i];
    }
    vec[k] = smem + q.vec[k];
  }
  __syncthreads();

  // One row of one tensor into its stage: its whole 16-byte units (bytes returned, issued
  // by thread 0) and, by the first threads, the elements at its ends.
  auto units = [&](const char* src, int size, int64_t* lo) {
    const int64_t at = reinterpret_cast<int64_t>(src);
    *lo = VEC ? at : (at + 15) & ~int64_t(15);
    const int64_t hi = VEC ? at + int64_t(d) * size : (at + int64_t(d) * size) & ~int64_t(15);
    return hi > *lo ? static_cast<uint32_t>(hi - *lo) : 0u;
  };
  auto ends = [&](const char* src, int size, char* stage) {
    if (VEC || tid >= 32) return;
    int64_t lo;
    const int64_t bytes = units(src, size, &lo), at = reinterpret_cast<int64_t>(src);
    const int head = bytes ? static_cast<int>(lo - at) / size : d;        // elements before the units
    const int tail = bytes ? static_cast<int>(lo + bytes - at) / size : d;  // first element behind them
    for (int i = tid; i < head + (d - tail); i += 32) {
      const int64_t e = int64_t(i < head ? i : tail + i - head) * size;
      char* dst = stage + (at & 15) + e;
      if (size == 4) *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src + e);
      else *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src + e);
    }
  };
  auto source = [&](const void* p, int dt, int64_t stride, int64_t i) {
    return static_cast<const char*>(row_of(p, dt, (blockIdx.x + i * gridDim.x) * stride));
  };
  auto bulk = [&](const char* src, int size, char* stage, uint64_t* bar) {
    int64_t lo;
    const uint32_t bytes = units(src, size, &lo);
    if (bytes) sm100::bulk_load(stage + (reinterpret_cast<int64_t>(src) & 15) + (lo - reinterpret_cast<int64_t>(src)),
                                reinterpret_cast<const void*>(lo), bytes, bar);
  };
  auto fill_y = [&](int64_t i) {                           // the CTA's row i
    if (!a.y || i >= n_rows) return;
    const int s = static_cast<int>(i % q.stages), size = a.y_dt == WUSH_FP32 ? 4 : 2;
    const char* src = source(a.y, a.y_dt, a.y_stride, i);
    char* stage = smem + q.y + s * q.y_step;
    if (tid == 0) {
      int64_t lo;
      sm100::mbar_arrive_expect_tx(&full[0][s], units(src, size, &lo));
      bulk(src, size, stage, &full[0][s]);
    }
    ends(src, size, stage);
  };
  auto fill_rest = [&](int64_t i) {
    if (i >= n_rows) return;
    const int s = static_cast<int>(i % q.stages);
    const int r_size = a.r_dt == WUSH_FP32 ? 4 : 2, g_size = a.gate_dt == WUSH_FP32 ? 4 : 2;
    const bool with_r = a.r && q.r >= 0, with_g = gate_rows && q.gate >= 0;
    const char* src_r = with_r ? source(a.r, a.r_dt, a.r_stride, i) : nullptr;
    const char* src_g = with_g ? source(a.gate, a.gate_dt, a.gate_stride, i) : nullptr;
    char* stage_r = smem + q.r + s * q.r_step;
    char* stage_g = smem + q.gate + s * q.gate_step;
    if (tid == 0) {
      int64_t lo;
      sm100::mbar_arrive_expect_tx(&full[1][s], (with_r ? units(src_r, r_size, &lo) : 0u) +
                                                    (with_g ? units(src_g, g_size, &lo) : 0u));
      if (with_r) bulk(src_r, r_size, stage_r, &full[1][s]);
      if (with_g) bulk(src_g, g_size, stage_g, &full[1][s]);
    }
    if (with_r) ends(src_r, r_size, stage_r);
    if (with_g) ends(src_g, g_size, stage_g);
  };
  // (a wait that gives up marks the error and lets the CTA run on, so that its barriers
  // stay uniform; every later wait then gives up at once)
  bool gave_up = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!sm100::mbar_wait_bounded(bar, parity, kDefaultPolls, kDeadlineNs, &abort_flag)) {
      *static_cast<volatile int*>(&abort_flag) = 1;
      gave_up = true;
    }
  };

  for (int64_t i = 0; i < q.stages; ++i) {
    fill_y(i);
    fill_rest(i);
  }
  for (int64_t i = 0; i < n_rows; ++i) {
    const int s = static_cast<int>(i % q.stages);
    const uint32_t parity = static_cast<uint32_t>(i / q.stages) & 1u;
    const int64_t row = blockIdx.x + i * gridDim.x;
    float (*sums)[32] = red[i & 1];
    float v[NV][8];
    auto phase = [&](const void* p, int dt, int64_t stride) {
      return VEC ? 0 : static_cast<int>(reinterpret_cast<int64_t>(row_of(p, dt, row * stride)) & 15);
    };
    auto r_row = [&]() -> const void* {
      return q.r >= 0 ? smem + q.r + s * q.r_step + phase(a.r, a.r_dt, a.r_stride)
                      : row_of(a.r, a.r_dt, row * a.r_stride);
    };
    if (!VEC) __syncthreads();                             // the rows' ends are in place
    if (a.y) {
      wait(&full[0][s], parity);
      load_row<VEC, NV>(smem + q.y + s * q.y_step + phase(a.y, a.y_dt, a.y_stride), a.y_dt, g, tid, d, v);
      apply_norm<VEC, NV>(a, a.post, vec[0], vec[1], v, sums, g, tid, 0, d);
      if (a.post.kind == WUSH_ROWNORM_NONE) __syncthreads();
      fill_y(i + q.stages);
      wait(&full[1][s], parity);
      const void* gate = !gate_rows ? vec[4]
                         : q.gate >= 0 ? smem + q.gate + s * q.gate_step + phase(a.gate, a.gate_dt, a.gate_stride)
                                       : row_of(a.gate, a.gate_dt, row * a.gate_stride);
      gate_and_add<VEC, NV>(a, gate, a.r ? r_row() : nullptr, v, g, tid, d);
      if (a.r_out) store_row<VEC, NV>(row_of(a.r_out, a.r_dt, row * a.r_out_stride), a.r_dt, g, tid, d, v);
    } else {
      wait(&full[1][s], parity);
      load_row<VEC, NV>(r_row(), a.r_dt, g, tid, d, v);
    }
    if (a.h) apply_norm<VEC, NV>(a, a.pre, vec[2], vec[3], v, sums + 2, g, tid, 0, d);
    if (!a.h || a.pre.kind == WUSH_ROWNORM_NONE) __syncthreads();
    fill_rest(i + q.stages);
    if (a.h) store_row<VEC, NV>(row_of(a.h, a.h_dt, row * a.h_stride), a.h_dt, g, tid, d, v);
  }
  if (gave_up) {
    atomicOr(&g_norm_error, kErrTimeoutBarrier);
    const uint64_t until = sm100::globaltimer_ns() + 200000ull;   // copies in flight may still land here
    while (sm100::globaltimer_ns() < until) __nanosleep(1000);
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

constexpr int kSmemPerSm = 224 * 1024;                     // what the rings of an SM's CTAs share
constexpr int kCtaOverhead = 3 * 1024;                     // static and reserved shared memory of a CTA

// The ring kernel's layout for ``ctas`` CTAs an SM: the shared memory it takes, or 0
// where not even one stage of y (or, without y, of x) fits.
int plan(const Args& a, bool vec, int ctas, int want_stages, Ring* q) {
  const int budget = kSmemPerSm / ctas - kCtaOverhead;
  auto up = [](int64_t n) { return static_cast<int>((n + 15) / 16 * 16); };
  const bool gate_rows = a.gate && a.gate_stride;
  const int edge = vec ? 0 : 16;                           // rows keep their 16-byte phase
  const int y = a.y ? up(int64_t(a.d) * dtype_bytes(a.y_dt) + edge) : 0;
  int r = a.r ? up(int64_t(a.d) * dtype_bytes(a.r_dt) + edge) : 0;
  int gate = gate_rows ? up(int64_t(a.d) * dtype_bytes(a.gate_dt) + edge) : 0;
  if (gate && y + r + gate > budget) gate = 0;             // rows too wide: read where they lie
  if (y && y + r + gate > budget) r = 0;
  if (y + r + gate > budget) return 0;
  const void* vecs[5] = {a.post.w, a.post.b, a.pre.w, a.pre.b, gate_rows ? nullptr : a.gate};
  const int dts[5] = {a.post.dt, a.post.dt, a.pre.dt, a.pre.dt, a.gate_dt};
  int all = 0;
  for (int k = 0; k < 5; ++k) all += vecs[k] ? up(int64_t(a.d) * dtype_bytes(dts[k])) : 0;
  const int stage = y + r + gate > 0 ? y + r + gate : 16;
  // vectors that leave no room for the stages stay where they are (in L2)
  const bool keep = q->kept = all + want_stages * stage <= budget;
  q->stages = (budget - (keep ? all : 0)) / stage;
  if (q->stages > kMaxStages) q->stages = kMaxStages;
  int at = 0;
  q->y = at; q->y_step = y; at += y * q->stages;
  q->r = r ? at : -1; q->r_step = r; at += r * q->stages;
  q->gate = gate ? at : -1; q->gate_step = gate; at += gate * q->stages;
  for (int k = 0; k < 5; ++k) {
    q->vec[k] = keep && vecs[k] ? at : -1;
    if (q->vec[k] >= 0) at += up(int64_t(a.d) * dtype_bytes(dts[k]));
  }
  return at > 16 ? at : 16;
}

template <bool VEC, int NV, int G>
int launch_ring(const Args& a, int sms, cudaStream_t st) {
  Ring q = {};
  // As many CTAs an SM as leave each two stages and the vectors (while one CTA waits in
  // its reductions the others use the memory); where rows are too wide for that, two
  // stages without the vectors, then what fits.
  constexpr int kMost = 1024 / G;                          // (64 registers a thread)
  int ctas = kMost, smem = 0;
  while (ctas > 0 && !((smem = plan(a, VEC, ctas, 2, &q)) && q.kept && q.stages >= 2)) --ctas;
  if (ctas == 0)
    for (ctas = kMost; ctas > 1 && !((smem = plan(a, VEC, ctas, 2, &q)) && q.stages >= 2);) --ctas;
  if (ctas == 1) smem = plan(a, VEC, 1, q.kept && q.stages >= 2 ? 2 : 1, &q);
  if (!smem) return WUSH_ERR_UNSUPPORTED;
  auto kern = norm_ring_kernel<VEC, NV, G>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, kSmemPerSm, done) != WUSH_OK) return WUSH_ERR_CUDA;
  const int64_t grid = int64_t(ctas) * sms < a.rows ? int64_t(ctas) * sms : a.rows;
  kern<<<static_cast<unsigned>(grid), G, smem, st>>>(a, q);
  return launch_status();
}

// Threads of a row and elements of a thread: up to 32 elements, and as few threads as
// hold the row then, since a reduction's cost grows with its warps.
template <bool VEC>
int launch_width(const Args& a, int sms, cudaStream_t st) {
  const int per128 = (a.d + 1023) / 1024;
  if (per128 == 1) return launch_ring<VEC, 1, 128>(a, sms, st);
  if (per128 == 2) return launch_ring<VEC, 2, 128>(a, sms, st);
  if (per128 <= 4) return launch_ring<VEC, 2, 256>(a, sms, st);
  if (per128 <= 6) return launch_ring<VEC, 3, 256>(a, sms, st);
  if (per128 <= 8) return launch_ring<VEC, 4, 256>(a, sms, st);
  if (per128 <= 12) return launch_ring<VEC, 3, 512>(a, sms, st);
  if (per128 <= 16) return launch_ring<VEC, 4, 512>(a, sms, st);
  return launch_ring<VEC, 4, 1024>(a, sms, st);
}

int round_up(int n, int m) { return (n + m - 1) / m * m; }

int run(Args& a, bool vec, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return WUSH_ERR_CUDA;
  const int groups = (a.d + 7) / 8;
  a.inv_d = 1.0f / static_cast<float>(a.d);
  // Few rows: the ring's set-up would cost more than it hides.
  if (a.rows <= 2 * sms && groups <= 1024) {
    int threads = round_up(groups, 32);
    if (threads < kMinThreads) threads = threads <= 32 ? 32 : threads <= 64 ? 64 : kMinThreads;
    a.row_threads = threads;
    const int block = threads < kMinThreads ? kMinThreads : threads;
    const int64_t per = block / threads, grid = (a.rows + per - 1) / per;
    if (vec) norm_few_kernel<true><<<static_cast<unsigned>(grid), block, 0, st>>>(a);
    else norm_few_kernel<false><<<static_cast<unsigned>(grid), block, 0, st>>>(a);
    return launch_status();
  }
  return vec ? launch_width<true>(a, sms, st) : launch_width<false>(a, sms, st);
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
