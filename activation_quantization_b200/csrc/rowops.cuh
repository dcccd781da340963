// What the operators around a quantised projection share: element types, their
// conversions, and the host checks on overlapping rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace wush {

inline int dtype_bytes(int dt) { return dt == WUSH_FP32 ? 4 : 2; }
inline bool known_dtype(int dt) { return dt == WUSH_BF16 || dt == WUSH_FP32 || dt == WUSH_FP16; }

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

// One element.
__device__ __forceinline__ float load1(const void* p, int dt, int64_t i) {
  if (dt == WUSH_FP32) return static_cast<const float*>(p)[i];
  if (dt == WUSH_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
// (each output is rounded once, to nearest even; fp16 beyond its range becomes an infinity)
__device__ __forceinline__ void store1(void* p, int dt, int64_t i, float v) {
  if (dt == WUSH_FP32) static_cast<float*>(p)[i] = v;
  else if (dt == WUSH_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Eight consecutive elements from a 16-byte boundary.
__device__ __forceinline__ void load8(const void* p, int dt, int64_t i, float (&v)[8]) {
  if (dt == WUSH_FP32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
  const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if (dt == WUSH_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) { v[2 * k] = bf16_lo(w[k]); v[2 * k + 1] = bf16_hi(w[k]); }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      v[2 * k] = f.x; v[2 * k + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void store8(void* p, int dt, int64_t i, const float (&v)[8]) {
  if (dt == WUSH_FP32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (dt == WUSH_BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 b = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace wush
