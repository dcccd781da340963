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
//  * few rows, or narrow ones: one CTA a row (narrow rows share one), loads straight to
//    registers (latency counts);
//  * many rows: persistent CTAs, each with a ring of whole rows in shared memory that
//    bulk copies fill ahead of it, so that the bytes in flight do not depend on how
//    many threads wait.  4096 rows x 4096, fp32 y, bf16 stream and h: 29.2 us, 5.75 TB/s;
//    8192 x 5120 bf16, the norm alone: 30.6 us, 5.48 TB/s; 2048 x 12288 fp32 with layer
//    norms and a gate per element: 90 us, 5.04 TB/s (its four vectors do not fit beside
//    the rows and are read from L2 for each row); 1531 x 4097 bf16 with a gate per element, rows
//    at any element: 23.9 us, 2.62 TB/s (199 of the 444 CTAs have four rows, the others three).
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
constexpr int64_t kFewRows = 296;                           // two a SM
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
  int64_t rows, polls;                                     // polls: see kDefaultPolls
  int d, row_threads;                                      // threads of one row (a multiple of 32)
  float inv_d;
  int phase, phase_step;                                   // kShifted: row i begins (phase + i phase_step) % 4 behind a quad
  bool mute;                                               // test hook: the ring's rows are not asked for
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

// The exponential is 2^t with t = -g log2 e rounded to fp32, the quotient within 2 ulp: some
// (10 + |g|) 2^-24 of the result, which outputs of 16 bits do not see.  With expf and a rounded reciprocal
// instead, 4096 rows x 5120 with a gate per channel take 54.0 us (44.6 so), 1531 x 4097 with a gate per
// element 28.9 (23.6), 8192 x 1024 31.4 (24.7); with expf alone 48.2, 24.4 and 29.4.
__device__ __forceinline__ float activate(float g, int act) {
  if (act == WUSH_GATE_LINEAR) return g;
  const float s = __fdividef(1.0f, 1.0f + __expf(-g));     // (0 where the sum is above 2^126)
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

// A norm's vectors: in shared memory as fp32, the weight with its offset added
// (``staged``), or where the caller has them.
struct Vectors {
  bool staged;
  const float* w;
  const float* b;
};

// v = N(v) over the row.
template <int MODE, int NV>
__device__ __forceinline__ void apply_norm(const Args& a, const NormArgs& n, const Vectors& vec, float (&v)[NV][8],
                                           float (*red)[32], const Columns<MODE>& q, int warp0) {
  if (n.kind == WUSH_ROWNORM_NONE) return;
  const int warps = q.g >> 5;
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
      for (int e = 0; e < 8; ++e) {
        const int c = MODE == kScalar ? q.at(j, e) : q.at(j, e & 4);     // (a quad's first column speaks for it)
        v[j][e] = c < q.d ? v[j][e] - mean : 0.0f;
      }
    mask_edges<MODE, NV>(q, v);
  }
  float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j) sq = squares8(v[j], sq);
  const float f = rsqrtf(fmaf(row_sum(sq.x + sq.y, red[1], warps, warp0), a.inv_d, n.eps));
  if (vec.staged && vec.w) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      load_group<WUSH_FP32, MODE>(vec.w, j, q, x);
      scale8(v[j], f);
      mul8(v[j], x);
    }
  } else if (MODE != kShifted && n.w) {
    with_dtype(n.dt, [&](auto dt) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<dt.value, MODE>(n.w, j, q, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += n.offset;
        scale8(v[j], f);
        mul8(v[j], x);
      }
    });
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) scale8(v[j], f);
  }
  if (vec.staged && vec.b) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      load_group<WUSH_FP32, MODE>(vec.b, j, q, x);
      add8(v[j], x);
    }
  } else if (MODE != kShifted && n.b) {
    with_dtype(n.dt, [&](auto dt) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<dt.value, MODE>(n.b, j, q, x);
        add8(v[j], x);
      }
    });
  }
}

template <int MODE, int NV>
__device__ __forceinline__ void load_row(const void* row, int dt, const Columns<MODE>& q, float (&v)[NV][8]) {
  with_dtype(dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_group<t.value, MODE>(row, j, q, v[j]);
  });
  mask_edges<MODE, NV>(q, v);
}

template <int MODE, int NV>
__device__ __forceinline__ void store_row(void* row, int dt, const Columns<MODE>& q, const float (&v)[NV][8]) {
  with_dtype(dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NV; ++j) store_group<t.value, MODE>(row, j, q, v[j]);
  });
}

// v = residual_scale * r + branch_scale * v * act(gate).
template <int MODE, int NV>
__device__ __forceinline__ void gate_and_add(const Args& a, const void* gate, int gate_dt, const void* r,
                                             float (&v)[NV][8], const Columns<MODE>& q) {
  if (gate)
    with_dtype(gate_dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<t.value, MODE>(gate, j, q, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= activate(x[e], a.act);
      }
    });
  if (r) {
    with_dtype(a.r_dt, [&](auto t) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        load_group<t.value, MODE>(r, j, q, x);
        blend8(v[j], a.branch_scale, x, a.residual_scale);
      }
    });
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) scale8(v[j], a.branch_scale);
  }
  mask_edges<MODE, NV>(q, v);
}

// ---------------------------------------------------------------------------
// Few or narrow rows: one CTA a row, narrow rows sharing one.
// ---------------------------------------------------------------------------
template <int MODE>
__global__ void __launch_bounds__(1024) norm_few_kernel(const __grid_constant__ Args a) {
  __shared__ __align__(16) float red[4][32];
  const int g = a.row_threads, sub = threadIdx.x / g, tid = threadIdx.x - sub * g, warp0 = sub * (g >> 5);
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / g) + sub;
  const bool live = row < a.rows;                          // the others only take part in the barriers
  const Columns<MODE> q = {g, tid, live ? a.d : 0, 0, false};
  float v[1][8];
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const void* r = a.r ? row_of(a.r, a.r_dt, row * a.r_stride) : nullptr;
  if (a.y) {
    load_row<MODE, 1>(row_of(a.y, a.y_dt, row * a.y_stride), a.y_dt, q, v);
    apply_norm<MODE, 1>(a, a.post, Vectors{}, v, red, q, warp0);
    gate_and_add<MODE, 1>(a, a.gate ? row_of(a.gate, a.gate_dt, row * a.gate_stride) : nullptr, a.gate_dt, r, v, q);
    if (a.r_out) store_row<MODE, 1>(row_of(a.r_out, a.r_dt, row * a.r_out_stride), a.r_dt, q, v);
  } else {
    load_row<MODE, 1>(r, a.r_dt, q, v);
  }
  if (a.h) {
    apply_norm<MODE, 1>(a, a.pre, Vectors{}, v, red + 2, q, warp0);
    store_row<MODE, 1>(row_of(a.h, a.h_dt, row * a.h_stride), a.h_dt, q, v);
  }
}

// ---------------------------------------------------------------------------
// Many rows: a ring of rows in shared memory.
//
// A stage of a tensor holds one row at the 16-byte phase that the row has in global
// memory, so that a bulk copy of the 16-byte units that it touches brings it.  y has a
// barrier of its own, r and the gate share one: y's stage is refilled as soon as the
// first reduction has read it, the others' after the second.
// ---------------------------------------------------------------------------
// CTAs an SM: 64 registers a thread, 80 where a thread of 256 has more than 16 elements.  With 32 elements
// a thread spills at 64 (some 200 bytes, 400 in single elements).  One CTA fewer, which does not, measured at
// 2048 rows: 16384 wide, fp32 y, RMS norms 60.5 us (57.0 so), layer norms with gate in fp32 117.9 (137.7), the
// norm alone 27.2 (35.2); 8192 wide, two of 256 threads: 30.9 (31.8), 59.1 (66.0), 15.8 (18.0).
constexpr int ring_ctas(int nv, int g) { return g == 256 && nv > 2 ? 3 : 1024 / g; }

template <int MODE, int NV, int G>
__global__ void __launch_bounds__(G, ring_ctas(NV, G)) norm_ring_kernel(const __grid_constant__ Args a,
                                                         const __grid_constant__ Ring q) {
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) float red[2][4][32];
  __shared__ __align__(8) uint64_t full[2][kMaxStages];    // [y | r and gate]
  __shared__ int abort_flag;
  constexpr int g = G;                                     // (a constant, so that columns are immediate offsets)
  const int tid = threadIdx.x, d = a.d;
  // (a CTA's rows are gridDim.x apart, a multiple of four, and so all have one shift)
  Columns<MODE> cols = {g, tid, d, MODE == kShifted ? (a.phase + static_cast<int>(blockIdx.x & 3) * a.phase_step) & 3 : 0,
                        false};
  if (MODE == kShifted) cols.edges = cols.find_edges(NV);
  const bool gate_rows = a.gate && a.gate_stride, gate_ring = gate_rows && q.gate >= 0, r_ring = a.r && q.r >= 0;
  const int lane = tid & 31;
  const int n_rows = static_cast<int>((a.rows - 1 - blockIdx.x) / gridDim.x) + 1;   // (at most one CTA a row)

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&full[0][i], 1);
      mbar_init(&full[1][i], gate_ring ? 2 : 1);
    }
    sm100::fence_barrier_init();
  }
  for (int i = tid; i < 2 * 4 * 32; i += g) (&red[0][0][0])[i] = 0.0f;
  sm100::pdl_wait();                                       // nothing global is touched before this
  sm100::pdl_launch_dependents();
  __syncthreads();                                         // the barriers are set up
  // One row of one tensor into its stage, by a bulk copy of the 16-byte units that it touches:
  // ``units`` gives their first byte and their number of bytes.  Each tensor has a warp for it (y
  // the third, r the first, the gate the second), since the slowest warp holds up the row.  What a unit holds
  // beside the row is never used.  Units that reach beyond the matrix (its first row's first,
  // its last row's last) are left out, and the warp copies the elements there.
  struct Bounds {
    int64_t lo, hi;                                        // the matrix's whole units
  };
  auto bounds = [&](const void* p, int dt, int64_t stride) {
    const int64_t at = reinterpret_cast<int64_t>(p);
    return Bounds{(at + 15) & ~int64_t(15),
                  reinterpret_cast<int64_t>(row_of(p, dt, (a.rows - 1) * stride + d)) & ~int64_t(15)};
  };
  struct Units {
    int64_t lo;
    uint32_t bytes;
  };
  auto units = [&](int64_t at, int size, const Bounds& m) {
    const int64_t end = at + int64_t(d) * size;
    if (MODE == kAligned) return Units{at, static_cast<uint32_t>(end - at)};
    const int64_t from = at & ~int64_t(15), to = (end + 15) & ~int64_t(15), hi = to < m.hi ? to : m.hi;
    const int64_t lo = from > m.lo ? from : m.lo;
    return Units{lo, hi > lo ? static_cast<uint32_t>(hi - lo) : 0u};
  };
  auto bulk = [&](int64_t at, const Units& u, char* to, uint64_t* bar) {
    if (u.bytes) sm100::bulk_load(to + (at & 15) + (u.lo - at), reinterpret_cast<const void*>(u.lo), u.bytes, bar);
  };
  auto ends = [&](int64_t at, int size, const Units& u, char* to) {
    const int64_t hi = u.lo + u.bytes, end = at + int64_t(d) * size;
    if (u.bytes && u.lo <= at && hi >= end) return;
    const int head = !u.bytes ? d : u.lo > at ? static_cast<int>(u.lo - at) / size : 0;   // elements before the units
    const int tail = !u.bytes ? d : hi < end ? static_cast<int>(hi - at) / size : d;      // first element behind them
    for (int i = lane; i < head + (d - tail); i += 32) {
      const int e = (i < head ? i : tail + i - head) * size;
      char* dst = to + (at & 15) + e;
      if (size == 4) *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(at + e);
      else *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(at + e);
    }
  };
  const Bounds in_y = bounds(a.y, a.y_dt, a.y_stride), in_r = bounds(a.r, a.r_dt, a.r_stride),
               in_g = bounds(a.gate, a.gate_dt, a.gate_stride);
  auto address = [&](const void* p, int dt, int64_t stride, int i) {       // of the CTA's row i
    return reinterpret_cast<int64_t>(row_of(p, dt, (blockIdx.x + int64_t(i) * gridDim.x) * stride));
  };
  const int y_size = a.y_dt == WUSH_FP32 ? 4 : 2, r_size = a.r_dt == WUSH_FP32 ? 4 : 2,
            gate_size = a.gate_dt == WUSH_FP32 ? 4 : 2;
  auto fill = [&](const void* p, int dt, int64_t stride, int size, const Bounds& in, int i, char* to, uint64_t* bar) {
    const int64_t at = address(p, dt, stride, i);          // (by one warp, its first thread where no ends are left)
    const Units u = units(at, size, in);
    if (lane == 0) {
      sm100::mbar_arrive_expect_tx(bar, u.bytes);
      bulk(at, u, to, bar);
    }
    if (MODE != kAligned) ends(at, size, u, to);
  };
  const int role = MODE == kAligned && lane ? -1 : tid >> 5;
  // (a thread that has given up a wait asks for nothing more: its stages' turns are not over)
  int n_fill = a.mute ? 0 : n_rows;
  auto fill_y = [&](int i, int s) {                        // the CTA's row i into stage s
    if (a.y && i < n_fill && role == 2) fill(a.y, a.y_dt, a.y_stride, y_size, in_y, i, smem + q.y + s * q.y_step, &full[0][s]);
  };
  auto fill_rest = [&](int i, int s) {
    if (i >= n_fill) return;
    if (role == 0) {
      if (r_ring) fill(a.r, a.r_dt, a.r_stride, r_size, in_r, i, smem + q.r + s * q.r_step, &full[1][s]);
      else if (lane == 0) sm100::mbar_arrive_expect_tx(&full[1][s], 0);
    } else if (role == 1 && gate_ring) {
      fill(a.gate, a.gate_dt, a.gate_stride, gate_size, in_g, i, smem + q.gate + s * q.gate_step, &full[1][s]);
    }
  };
  // (a wait that gives up marks the error and lets the CTA run on, so that its barriers
  // stay uniform; every later wait then gives up soon)
  bool gave_up = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (sm100::mbar_try_wait(bar, parity) || gave_up) return;
    if (!sm100::mbar_wait_bounded(bar, parity, a.polls, kDeadlineNs, &abort_flag)) {
      *static_cast<volatile int*>(&abort_flag) = 1;
      gave_up = true;
      n_fill = 0;
    }
  };

  for (int i = 0; i < q.stages; ++i) {
    fill_y(i, i);
    fill_rest(i, i);
  }
  // Meanwhile the vectors that every row uses, as fp32 and shifted like the rows; eight elements of
  // each are asked for before any is stored; shifted ones go to the threads one by one, so that a
  // warp's lie side by side on both sides.
  Vectors post = {q.kept, nullptr, nullptr}, pre = post;
  const float* gate_vec = nullptr;
  if (q.kept) {
    const void* src[5] = {a.post.w, a.post.b, a.pre.w, a.pre.b, gate_rows ? nullptr : a.gate};
    const int dts[5] = {a.post.dt, a.post.dt, a.pre.dt, a.pre.dt, a.gate_dt};
    const float offset[5] = {a.post.offset, 0.0f, a.pre.offset, 0.0f, 0.0f};
    float* dst[5];
#pragma unroll
    for (int n = 0; n < 5; ++n) dst[n] = src[n] ? reinterpret_cast<float*>(smem + q.vec[n]) + cols.shift : nullptr;
    if constexpr (MODE == kAligned) {
      // whether all vectors have one type (that of an absent one says nothing)
      const bool has_post = src[0] || src[1], has_pre = src[2] || src[3];
      const bool alike = (!has_post || !has_pre || dts[0] == dts[2]) &&
                         (!src[4] || ((!has_pre || dts[4] == dts[2]) && (!has_post || dts[4] == dts[0])));
#pragma unroll 1
      for (int j = 0; j < NV; ++j) {
        float x[5][8];
        if (alike) {
          with_dtype(src[4] ? dts[4] : has_pre ? dts[2] : dts[0], [&](auto t) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < 5; ++n)
              if (src[n]) load_group<t.value, kAligned>(src[n], j, cols, x[n]);
          });
        } else {
#pragma unroll
          for (int n = 0; n < 5; ++n)
            if (src[n])
              with_dtype(dts[n], [&](auto t) __attribute__((always_inline)) {
                load_group<t.value, kAligned>(src[n], j, cols, x[n]);
              });
        }
#pragma unroll
        for (int n = 0; n < 5; ++n)
          if (src[n])
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = cols.at(j, e);
              if (cols.has(c)) dst[n][c] = x[n][e] + offset[n];
            }
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < NV; ++j) {
        uint32_t w[5][8];                                    // the vectors' bytes; converted once all are asked for
#pragma unroll
        for (int n = 0; n < 5; ++n) {
          if (!src[n]) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) w[n][e] = 0u;
          if (dts[n] == WUSH_FP32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = (j * 8 + e) * g + tid;
              if (c < d) w[n][e] = static_cast<const uint32_t*>(src[n])[c];
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = (j * 8 + e) * g + tid;
              if (c < d) w[n][e] = static_cast<const uint16_t*>(src[n])[c];
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 5; ++n)
          if (src[n])
            with_dtype(dts[n], [&](auto t) __attribute__((always_inline)) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int c = (j * 8 + e) * g + tid;
                const float x = t.value == WUSH_FP32   ? __uint_as_float(w[n][e])
                                : t.value == WUSH_BF16 ? bf16_lo(w[n][e])
                                                       : __half2float(__ushort_as_half(static_cast<unsigned short>(w[n][e])));
                if (c < d) dst[n][c] = x + offset[n];
              }
            });
      }
    }
    post.w = dst[0]; post.b = dst[1];
    pre.w = dst[2]; pre.b = dst[3];
    gate_vec = dst[4];
    __syncthreads();
  }
  int s = 0;
  uint32_t parity = 0;
  for (int i = 0; i < n_rows; ++i) {
    const int64_t row = blockIdx.x + int64_t(i) * gridDim.x;
    float (*sums)[32] = red[i & 1];
    float v[NV][8];
    // a row lies in its stage at the 16-byte phase that it has in global memory
    auto phase = [&](const void* p, int dt, int64_t stride) {
      return MODE == kAligned ? 0 : static_cast<int>(reinterpret_cast<int64_t>(row_of(p, dt, row * stride)) & 15);
    };
    const char* r_stage = smem + q.r + s * q.r_step + phase(a.r, a.r_dt, a.r_stride);
    if (MODE != kAligned) __syncthreads();                             // the rows' ends are in place
    if (a.y) {
      wait(&full[0][s], parity);
      load_row<MODE, NV>(smem + q.y + s * q.y_step + phase(a.y, a.y_dt, a.y_stride), a.y_dt, cols, v);
      apply_norm<MODE, NV>(a, a.post, post, v, sums, cols, 0);
      if (a.post.kind == WUSH_ROWNORM_NONE) __syncthreads();
      fill_y(i + q.stages, s);
      wait(&full[1][s], parity);
      const void* gate = nullptr;
      int gate_dt = a.gate_dt;
      if (gate_ring) gate = smem + q.gate + s * q.gate_step + phase(a.gate, a.gate_dt, a.gate_stride);
      else if (gate_vec) gate = gate_vec, gate_dt = WUSH_FP32;
      else if (a.gate) gate = row_of(a.gate, a.gate_dt, row * a.gate_stride);
      gate_and_add<MODE, NV>(a, gate, gate_dt,
                             r_ring ? r_stage : a.r ? row_of(a.r, a.r_dt, row * a.r_stride) : nullptr, v, cols);
      if (a.r_out) store_row<MODE, NV>(row_of(a.r_out, a.r_dt, row * a.r_out_stride), a.r_dt, cols, v);
    } else {
      wait(&full[1][s], parity);
      load_row<MODE, NV>(r_stage, a.r_dt, cols, v);
    }
    if (a.h) apply_norm<MODE, NV>(a, a.pre, pre, v, sums + 2, cols, 0);
    if (!a.h || a.pre.kind == WUSH_ROWNORM_NONE) __syncthreads();
    fill_rest(i + q.stages, s);
    if (a.h) store_row<MODE, NV>(row_of(a.h, a.h_dt, row * a.h_stride), a.h_dt, cols, v);
    if (++s == q.stages) s = 0, parity ^= 1;
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

// Whether an output's rows share a byte with a vector of ``bytes`` (one that lies between two
// rows does not).
bool on_vector(const Span& out, int64_t rows, const void* vector, int64_t bytes) {
  const char* v = static_cast<const char*>(vector);
  if (!out.p || !v || v >= out.p + (rows - 1) * out.stride + out.width || out.p >= v + bytes) return false;
  const int64_t behind = ((v - out.p) % out.stride + out.stride) % out.stride;     // of a row's first byte
  return behind < out.width || behind + bytes > out.stride;
}

bool on_norm(const Span& out, int64_t rows, const NormArgs& n, int64_t d) {
  const int64_t bytes = d * dtype_bytes(n.dt);
  return on_vector(out, rows, n.w, bytes) || on_vector(out, rows, n.b, bytes);
}

constexpr int kSmemPerSm = 224 * 1024;                     // what the rings of an SM's CTAs share
constexpr int kCtaOverhead = 3 * 1024;                     // static and reserved shared memory of a CTA
constexpr int kInFlight = 96 * 1024;                       // bytes of rows that an SM asks for ahead

// The ring kernel's layout for ``ctas`` CTAs an SM, and the shared memory it takes.
//
// An SM needs some 50 KB in flight to fill its share of the memory's bandwidth; with as
// many CTAs as the registers allow, one stage each gives that for rows of 24 KB (a stage
// is refilled while its row is still being worked on in registers) and narrower rows take
// up to four.  Measured (before the programmatic launch took another 2 us off) at 4096 rows
// x 4096, fp32 y, bf16 stream: four CTAs of 256 threads with one stage 30.7 us, two with two
// stages 34.4 us, eight of 128 threads 32.5 us; at 8192 x 5120 bf16, three CTAs: 31.3 us with
// three stages, 33.1 us with two.
int plan(const Args& a, bool aligned, int ctas, Ring* q) {
  const int budget = kSmemPerSm / ctas - kCtaOverhead;
  auto up = [](int64_t n) { return static_cast<int>((n + 15) / 16 * 16); };
  const bool gate_rows = a.gate && a.gate_stride;
  const int edge = aligned ? 0 : 16;                           // rows keep their 16-byte phase
  const int y = a.y ? up(int64_t(a.d) * dtype_bytes(a.y_dt) + edge) : 0;
  int r = a.r ? up(int64_t(a.d) * dtype_bytes(a.r_dt) + edge) : 0;
  int gate = gate_rows ? up(int64_t(a.d) * dtype_bytes(a.gate_dt) + edge) : 0;
  if (gate && y + r + gate > budget) gate = 0;             // too wide: read where it lies
  if (y && y + r + gate > budget) r = 0;
  const int stage = y + r + gate > 16 ? y + r + gate : 16;
  q->stages = kInFlight / ctas / stage;
  if (q->stages < 1) q->stages = 1;
  if (q->stages > kMaxStages) q->stages = kMaxStages;
  const void* vecs[5] = {a.post.w, a.post.b, a.pre.w, a.pre.b, gate_rows ? nullptr : a.gate};
  int all = 0;
  for (int k = 0; k < 5; ++k) all += vecs[k] ? up(int64_t(a.d) * 4 + edge) : 0;
  q->kept = all + q->stages * stage <= budget;             // otherwise they are read from L2, row by row
  int at = 0;
  q->y = at; q->y_step = y; at += y * q->stages;
  q->r = r ? at : -1; q->r_step = r; at += r * q->stages;
  q->gate = gate ? at : -1; q->gate_step = gate; at += gate * q->stages;
  for (int k = 0; k < 5; ++k) {
    q->vec[k] = q->kept && vecs[k] ? at : -1;
    if (q->vec[k] >= 0) at += up(int64_t(a.d) * 4 + edge);
  }
  return at;
}

template <int MODE, int NV, int G>
int launch_ring(const Args& a, int sms, cudaStream_t st) {
  Ring q = {};
  int ctas = ring_ctas(NV, G), smem = plan(a, MODE == kAligned, ctas, &q);
  if (MODE == kShifted) {                                  // all in shared memory, with fewer CTAs if need be
    const bool gate_rows = a.gate && a.gate_stride;
    while (ctas > 1 && !(q.kept && (!a.r || q.r >= 0) && (!gate_rows || q.gate >= 0)))
      smem = plan(a, false, --ctas, &q);
    if (!(q.kept && (!a.r || q.r >= 0) && (!gate_rows || q.gate >= 0))) return WUSH_ERR_UNSUPPORTED;
  }
  auto kern = norm_ring_kernel<MODE, NV, G>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, kSmemPerSm, done) != WUSH_OK) return WUSH_ERR_CUDA;
  const int64_t most = int64_t(ctas) * sms / 4 * 4, grid = most < a.rows ? most : a.rows;
  return launch_pdl(kern, static_cast<unsigned>(grid), G, smem, st, a, q);
}

// Threads of a row: 256 with up to 32 elements each (320 with 16 where those hold the row: a
// third group for the last few columns would cost every thread), more for wide rows.
template <int MODE>
int launch_width(const Args& a, int sms, cudaStream_t st) {
  const int d = a.d + (MODE == kShifted ? 3 : 0);
  if (d <= 4096) return launch_ring<MODE, 2, 256>(a, sms, st);
  if (d <= 5120) return launch_ring<MODE, 2, 320>(a, sms, st);
  if (d <= 6144) return launch_ring<MODE, 3, 256>(a, sms, st);
  if (d <= 8192) return launch_ring<MODE, 4, 256>(a, sms, st);
  if (d <= 12288) return launch_ring<MODE, 3, 512>(a, sms, st);
  if (d <= 16384) return launch_ring<MODE, 4, 512>(a, sms, st);
  return launch_ring<MODE, 4, 1024>(a, sms, st);
}

// Whether every matrix's rows begin equally far behind a quad's boundary (Columns); the
// first row's distance and the step from row to row.
bool shifted(Args* a) {
  const struct { const void* p; int dt; int64_t stride; } m[5] = {
      {a->y, a->y_dt, a->y_stride}, {a->r, a->r_dt, a->r_stride},
      {a->gate_stride ? a->gate : nullptr, a->gate_dt, a->gate_stride},
      {a->r_out, a->r_dt, a->r_out_stride}, {a->h, a->h_dt, a->h_stride}};
  int phase = -1, step = 0;
  for (const auto& t : m) {
    if (!t.p) continue;
    const int at = static_cast<int>(reinterpret_cast<uintptr_t>(t.p) / dtype_bytes(t.dt) & 3);
    const int by = static_cast<int>(t.stride & 3);
    if (phase >= 0 && (at != phase || by != step)) return false;
    phase = at;
    step = by;
  }
  a->phase = phase;
  a->phase_step = step;
  return a->d + 3 <= kMaxWidth;
}

int round_up(int n, int m) { return (n + m - 1) / m * m; }

int run(Args& a, bool vec, cudaStream_t st) {
  const int groups = (a.d + 7) / 8;
  a.mute = g_wait_limit_override > 0;
  a.polls = a.mute ? g_wait_limit_override : kDefaultPolls;
  a.inv_d = 1.0f / static_cast<float>(a.d);
  // Few rows, or narrow ones: the ring's set-up would cost more than it hides, and a ring CTA's 256
  // threads have one row of up to 4096 columns at a time, however few it has.  Measured, the ring
  // second: 7696 rows of 174, 16 bits: 4.9 and 29 us; 5536 of 1216, fp32 y, layer norm, gate:
  // 24.9 and 35.5; fp32 y, bf16 stream, 4096 rows of 1024: 11.3 and 25.2, of 2048: 20.4 and 26.0;
  // 16384 rows of 2048: 69.5 and 82.8; 8192 of 2047, 16 bits, gate: 82.9 and 70.0; 4096 of 4096,
  // fp32 y: 38.7 and 29.0.
  if ((a.rows <= kFewRows && groups <= 1024) || groups <= 256) {
    int threads = round_up(groups, 32);
    if (threads < kMinThreads) threads = threads <= 32 ? 32 : threads <= 64 ? 64 : kMinThreads;
    a.row_threads = threads;
    const int block = threads < kMinThreads ? kMinThreads : threads;
    const int64_t per = block / threads, grid = (a.rows + per - 1) / per;
    return vec ? launch_pdl(norm_few_kernel<kAligned>, static_cast<unsigned>(grid), block, 0, st, a)
               : launch_pdl(norm_few_kernel<kScalar>, static_cast<unsigned>(grid), block, 0, st, a);
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return WUSH_ERR_CUDA;
  if (vec) return launch_width<kAligned>(a, sms, st);
  if (shifted(&a)) {
    const int rc = launch_width<kShifted>(a, sms, st);
    if (rc != WUSH_ERR_UNSUPPORTED) return rc;
  }
  return launch_width<kScalar>(a, sms, st);
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
    if (on_norm(out, rows, a.post, d) || on_norm(out, rows, a.pre, d)) return WUSH_ERR_INVALID_ARG;
    // (a gate per channel is one row, read by every row)
    if (q.gate_stride ? overlap(out, span(q.gate, q.gate_dtype, q.gate_stride, d), rows)
                      : on_vector(out, rows, q.gate, d * dtype_bytes(q.gate_dtype)))
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
  const Span sh = span(h, h_dtype, h_stride, d);
  if ((!in_place && overlap(sh, span(x, x_dtype, x_stride, d), rows)) || on_norm(sh, rows, a.pre, d))
    return WUSH_ERR_INVALID_ARG;
  a.r = x; a.r_dt = x_dtype; a.r_stride = x_stride;
  a.h = h; a.h_dt = h_dtype; a.h_stride = h_stride;
  a.rows = rows; a.d = static_cast<int>(d);
  return run(a, vec, static_cast<cudaStream_t>(stream));
}
