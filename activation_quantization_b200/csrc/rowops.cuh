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

// One element.
template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == WUSH_FP32) return static_cast<const float*>(p)[i];
  if (DT == WUSH_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// Eight elements of a row as one thread of G holds them.  VEC: two quads, 4 G apart, so
// that a warp's accesses are contiguous in every type (16 bytes a lane in fp32, 8 in
// 16 bits); columns at or beyond d (a multiple of 4) read as zero.  Otherwise eight
// single elements, G apart.
template <bool VEC>
__device__ __forceinline__ int group_column(int j, int e, int g, int tid) {
  return VEC ? ((2 * j + (e >> 2)) * g + tid) * 4 + (e & 3) : (j * 8 + e) * g + tid;
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_group(const void* row, int j, int g, int tid, int d, float (&v)[8]) {
  using T = typename std::conditional<DT == WUSH_FP32, float, uint16_t>::type;
  const T* p = static_cast<const T*>(row);
  auto convert = [](uint32_t u) {
    return DT == WUSH_BF16 ? bf16_lo(u) : __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
  };
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = group_column<true>(j, 4 * h, g, tid);
      if (DT == WUSH_FP32) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < d) q = *reinterpret_cast<const float4*>(p + c);
        v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
      } else {
        uint2 q = make_uint2(0u, 0u);
        if (c < d) q = *reinterpret_cast<const uint2*>(p + c);
        v[4 * h] = convert(q.x & 0xffffu); v[4 * h + 1] = convert(q.x >> 16);
        v[4 * h + 2] = convert(q.y & 0xffffu); v[4 * h + 3] = convert(q.y >> 16);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = group_column<false>(j, e, g, tid);
      if (DT == WUSH_FP32) v[e] = c < d ? static_cast<const float*>(row)[c] : 0.0f;
      else v[e] = convert(c < d ? static_cast<const uint16_t*>(row)[c] : 0u);
    }
  }
}

// Each element is rounded once, to nearest even (fp16 beyond its range becomes an
// infinity).
template <int DT, bool VEC>
__device__ __forceinline__ void store_group(void* row, int j, int g, int tid, int d, const float (&v)[8]) {
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
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = group_column<true>(j, 4 * h, g, tid);
      if (c >= d) continue;
      if (DT == WUSH_FP32)
        *reinterpret_cast<float4*>(static_cast<float*>(row) + c) =
            make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + c) = make_uint2(u[2 * h], u[2 * h + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = group_column<false>(j, e, g, tid);
      if (c >= d) continue;
      if (DT == WUSH_FP32) static_cast<float*>(row)[c] = v[e];
      else static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(e & 1 ? u[e / 2] >> 16 : u[e / 2]);
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
