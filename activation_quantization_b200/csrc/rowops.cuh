// What the operators around a quantised projection share: element types, their
// conversions, and the host checks on overlapping rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace wush {

// Error words of the kernels with bounded waits in block_norm.cu and lora.cu (see
// common.cuh).
int read_and_clear_norm_error(int* word);
int read_and_clear_lora_error(int* word);

inline int dtype_bytes(int dt) { return dt == WUSH_FP32 ? 4 : 2; }
inline bool known_dtype(int dt) { return dt == WUSH_BF16 || dt == WUSH_FP32 || dt == WUSH_FP16; }

// Launches with programmatic stream serialization: the kernel may be set up while the one
// before it ends, and waits for it (pdl_wait) before it touches global memory.  It lets its
// own dependents start (pdl_launch_dependents) only after that wait, so that whatever a
// dependent reads before its own wait is already complete.
template <typename... P, typename... A>
inline int launch_pdl(void (*kern)(P...), unsigned grid, int block, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return WUSH_ERR_CUDA;
  return launch_status();
}

struct Span {                                              // rows of a tensor, as bytes
  const char* p;
  int64_t stride, width;                                   // bytes
};

inline Span span(const void* p, int dt, int64_t stride, int64_t d) {
  return {static_cast<const char*>(p), stride * dtype_bytes(dt), d * dtype_bytes(dt)};
}

// Whether two sets of rows share a byte.  Rows of one stride can interleave (columns
// of one wide buffer); sets of unequal strides are kept apart as whole ranges.
inline bool overlap(const Span& a, const Span& b, int64_t rows) {
  if (!a.p || !b.p) return false;
  const char* a_end = a.p + (rows - 1) * a.stride + a.width;
  const char* b_end = b.p + (rows - 1) * b.stride + b.width;
  if (a_end <= b.p || b_end <= a.p) return false;
  if (a.stride != b.stride) return true;
  const int64_t delta = ((b.p - a.p) % a.stride + a.stride) % a.stride;
  return delta < a.width || a.stride - delta < b.width;
}

// Calls f with the element type as a compile-time constant, so that the branch lies
// outside the loops of f.
template <typename F>
__device__ __forceinline__ void with_dtype(int dt, F f) {
  if (dt == WUSH_BF16) f(std::integral_constant<int, WUSH_BF16>{});
  else if (dt == WUSH_FP32) f(std::integral_constant<int, WUSH_FP32>{});
  else f(std::integral_constant<int, WUSH_FP16>{});
}

// Two fp32 values at a time (sm_100's packed FMA pipe).
__device__ __forceinline__ void mul8(float (&v)[8], const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 p = __fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(x[e], x[e + 1]));
    v[e] = p.x; v[e + 1] = p.y;
  }
}
__device__ __forceinline__ void scale8(float (&v)[8], float f) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 p = __fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(f, f));
    v[e] = p.x; v[e + 1] = p.y;
  }
}
__device__ __forceinline__ void add8(float (&v)[8], const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 p = __fadd2_rn(make_float2(v[e], v[e + 1]), make_float2(x[e], x[e + 1]));
    v[e] = p.x; v[e + 1] = p.y;
  }
}
// v = f * v + g * x
__device__ __forceinline__ void blend8(float (&v)[8], float f, const float (&x)[8], float g) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 q = __fmul2_rn(make_float2(x[e], x[e + 1]), make_float2(g, g));
    const float2 p = __ffma2_rn(make_float2(v[e], v[e + 1]), make_float2(f, f), q);
    v[e] = p.x; v[e + 1] = p.y;
  }
}
__device__ __forceinline__ float2 squares8(const float (&v)[8], float2 s) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 p = make_float2(v[e], v[e + 1]);
    s = __ffma2_rn(p, p, s);
  }
  return s;
}

// How a row's elements go to the ``g`` threads that hold it, eight to a group.
//   kAligned:  every row of every matrix begins on a 16-byte boundary and d is a multiple of
//              8: two quads of elements a group, 4 g apart, so that a warp's accesses are
//              contiguous in every type (16 bytes a lane in fp32, 8 in 16 bits);
//   kShifted:  the rows begin at any element, but the same number (``shift``) of elements
//              behind a quad's boundary in every matrix, as in contiguous matrices of an odd
//              width: the same quads, begun ``shift`` columns before the row.  Quads that the
//              row fills in part are accessed by the element;
//   kScalar:   anything else: eight single elements, g apart.
enum : int { kScalar = 0, kShifted = 1, kAligned = 2 };

template <int MODE>
struct Columns {
  int g, tid, d, shift;
  bool edges;                                              // kShifted: the warp has quads that the row fills in part
  __device__ __forceinline__ int at(int j, int e) const {
    return MODE == kScalar ? (j * 8 + e) * g + tid
                           : ((2 * j + (e >> 2)) * g + tid) * 4 + (e & 3) - (MODE == kShifted ? shift : 0);
  }
  __device__ __forceinline__ bool has(int c) const { return (MODE != kShifted || c >= 0) && c < d; }
  // The same for all threads of a warp, for NV groups a thread.
  __device__ __forceinline__ bool find_edges(int nv) const {
    bool part = false;
    for (int j = 0; j < nv; ++j)
      for (int h = 0; h < 2; ++h) {
        const int c = at(j, 4 * h);
        part = part || (c < d && (c < 0 || c + 3 >= d));
      }
    return __any_sync(0xffffffffu, part);
  }
};

// Zeroes the elements of quads that the row does not have.
template <int MODE, int NV>
__device__ __forceinline__ void mask_edges(const Columns<MODE>& q, float (&v)[NV][8]) {
  if (MODE != kShifted || !q.edges) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = q.has(q.at(j, e)) ? v[j][e] : 0.0f;
}

// A group of a row; columns that the row does not have read as zero.  In kShifted the row
// lies in shared memory, where whole quads can be read at its ends, and their elements
// outside the row are whatever lies there (mask_edges).
template <int DT, int MODE>
__device__ __forceinline__ void load_group(const void* row, int j, const Columns<MODE>& q, float (&v)[8]) {
  using T = typename std::conditional<DT == WUSH_FP32, float, uint16_t>::type;
  const T* p = static_cast<const T*>(row);
  auto convert = [](uint32_t u) {
    return DT == WUSH_BF16 ? bf16_lo(u) : __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
  };
  if constexpr (MODE == kScalar) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = q.at(j, e);
      if (DT == WUSH_FP32) v[e] = q.has(c) ? static_cast<const float*>(row)[c] : 0.0f;
      else v[e] = convert(q.has(c) ? static_cast<const uint16_t*>(row)[c] : 0u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = q.at(j, 4 * h);
      if (DT == WUSH_FP32) {
        float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < q.d) u = *reinterpret_cast<const float4*>(p + c);
        v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
      } else {
        uint2 u = make_uint2(0u, 0u);
        if (c < q.d) u = *reinterpret_cast<const uint2*>(p + c);
        v[4 * h] = convert(u.x & 0xffffu); v[4 * h + 1] = convert(u.x >> 16);
        v[4 * h + 2] = convert(u.y & 0xffffu); v[4 * h + 3] = convert(u.y >> 16);
      }
    }
  }
}

// Each element is rounded once, to nearest even (fp16 beyond its range becomes an
// infinity).
template <int DT, int MODE>
__device__ __forceinline__ void store_group(void* row, int j, const Columns<MODE>& q, const float (&v)[8]) {
  uint32_t u[4];
  if (DT != WUSH_FP32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (DT == WUSH_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
  }
  auto one = [&](int e) {
    const int c = q.at(j, e);
    if (!q.has(c)) return;
    if (DT == WUSH_FP32) static_cast<float*>(row)[c] = v[e];
    else static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(e & 1 ? u[e / 2] >> 16 : u[e / 2]);
  };
  if (MODE == kScalar || (MODE == kShifted && q.edges)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) one(e);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = q.at(j, 4 * h);
      if (c >= q.d) continue;
      if (DT == WUSH_FP32)
        *reinterpret_cast<float4*>(static_cast<float*>(row) + c) =
            make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + c) = make_uint2(u[2 * h], u[2 * h + 1]);
    }
  }
}

// A row of a matrix of runtime type.
__device__ __forceinline__ const void* row_of(const void* p, int dt, int64_t offset) {
  return static_cast<const char*>(p) + offset * (dt == WUSH_FP32 ? 4 : 2);
}
__device__ __forceinline__ void* row_of(void* p, int dt, int64_t offset) {
  return static_cast<char*>(p) + offset * (dt == WUSH_FP32 ? 4 : 2);
}

}  // namespace wush
