// Low-rank adapters of many requests beside a shared projection:
//   y[t] = y_in[t] + scale[g] * B_g (A_g x[t]),   g = adapter[t].
//
// Tokens of one adapter are taken together, so that its matrices are read once for
// up to eight tokens.  Both products run as m16n8k16 MMAs with the adapter's matrix
// as the 16-row operand and the tokens as the 8 columns: the matrices go from global
// memory straight into MMA fragments (the order of k inside a step is free as long
// as both operands share it, so a lane takes 16 consecutive bytes of a row).
//
// Precision.  The products of 16-bit inputs are exact in fp32 and s = A x is kept in
// fp32; for the second product s is split into 16-bit terms whose sum carries at
// least 22 bits of it, so what rounds is the fp32 accumulation:
//   bf16: three bf16 terms (8 bits each, the range of fp32);
//   fp16: two fp16 terms (11 bits each) after a power-of-two scaling of the token's
//         s to below 1, undone exactly on the result.
#include <type_traits>

#include "rowops.cuh"
#include "sm100.cuh"

namespace wush {
namespace {

constexpr int kMaxRank = 256;
constexpr int64_t kMaxAdapters = 1 << 20, kMaxWidth = 1 << 24, kMaxTokens = 1 << 26;

struct LoraArgs {
  const void* x;
  const int32_t* adapter;
  const void* a;
  const void* b;
  const int32_t* ranks;
  const float* scale;
  const float* y_in;
  float* y;
  int64_t x_stride, y_in_stride, y_stride;
  int64_t tokens;
  int d_in, d_out, n_adapters, rank;
};

template <typename E>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<E, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename E>
struct Split;
template <>
struct Split<__nv_bfloat16> {
  static constexpr int kTerms = 3;
};
template <>
struct Split<__half> {
  static constexpr int kTerms = 2;
};

// The 16-bit terms of v; each is the nearest value to what the ones before it leave.
template <typename E>
__device__ __forceinline__ void split(float v, E (&t)[Split<E>::kTerms]) {
#pragma unroll
  for (int i = 0; i < Split<E>::kTerms; ++i) {
    if constexpr (std::is_same<E, __half>::value) {
      t[i] = __float2half_rn(v);
      v -= __half2float(t[i]);
    } else {
      t[i] = __float2bfloat16_rn(v);
      v -= __bfloat162float(t[i]);
    }
  }
}

// Power of two that brings values of largest magnitude ``top`` below 1, and its
// inverse; 1 where there is nothing to scale (zero, infinity, NaN).  The exponent is
// kept within what both factors can hold as normal numbers.
__device__ __forceinline__ void fp16_scaling(float top, float* down, float* up) {
  const int e = static_cast<int>((__float_as_uint(top) >> 23) & 0xff);     // top in [2^(e-127), 2^(e-126))
  *down = *up = 1.0f;
  if (e > 0 && e < 255) {
    const int s = e - 126 < -126 ? -126 : e - 126 > 126 ? 126 : e - 126;
    *down = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
    *up = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
  }
}

__device__ __forceinline__ uint32_t keep_below(uint32_t pair, int col, int k) {   // elements col, col + 1
  return col + 1 < k ? pair : col < k ? pair & 0xffffu : 0u;
}

// ---------------------------------------------------------------------------
// Few tokens: one cluster of eight CTAs takes up to eight tokens of one adapter
// through both products in one launch.
// ---------------------------------------------------------------------------
constexpr int kCluster = 8, kFewThreads = 256, kFewWarps = kFewThreads / 32;

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// MB: blocks of 16 ranks held at once.  Shared memory: the warps' partial s
// [8][MB * 16][8], this CTA's sum [MB * 16][8], the terms [kTerms][8][MB * 16 + 8].
template <typename E, int MB>
__global__ void __launch_bounds__(kFewThreads) lora_few_kernel(const __grid_constant__ LoraArgs p) {
  constexpr int kR = MB * 16, kT = Split<E>::kTerms, kRow = kR + 8;
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem);
  float* mine = part + kFewWarps * kR * 8;
  E* terms = reinterpret_cast<E*>(mine + kR * 8);
  __shared__ int s_tok[8], s_warp[kFewWarps];
  __shared__ float s_up[8];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = lane >> 2, c = lane & 3;
  const int cta = static_cast<int>(sm100::cluster_ctarank());
  const int64_t t = blockIdx.x / kCluster;
  const int g = p.adapter[t];
  const bool known = g >= 0 && g < p.n_adapters;
  int k = 0;
  if (known) {
    k = p.ranks ? p.ranks[g] : p.rank;
    k = k < 0 ? 0 : k > p.rank ? p.rank : k;
  }
  if (k == 0) {                                            // no adapter: y_in passes through
    if (p.y != p.y_in) {
      const float4* src = reinterpret_cast<const float4*>(p.y_in ? p.y_in + t * p.y_in_stride : nullptr);
      float4* dst = reinterpret_cast<float4*>(p.y + t * p.y_stride);
      for (int i = cta * kFewThreads + tid; i < p.d_out / 4; i += kCluster * kFewThreads)
        dst[i] = src ? src[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    return;
  }
  // The tokens of an adapter go in groups of eight in their order; the cluster of a
  // group's first token takes it, the others leave.  (All CTAs of a cluster decide alike.)
  int before = 0;
  for (int64_t i0 = 0; i0 < t; i0 += kFewThreads) {
    const int64_t i = i0 + tid;
    before += __syncthreads_count(i < t && p.adapter[i] == g);
  }
  if (before % 8) return;
  if (tid < 8) s_tok[tid] = tid == 0 ? static_cast<int>(t) : -1;
  int found = 1;
  for (int64_t i0 = t + 1; i0 < p.tokens && found < 8; i0 += kFewThreads) {
    const int64_t i = i0 + tid;
    const bool hit = i < p.tokens && p.adapter[i] == g;
    const uint32_t m = __ballot_sync(0xffffffffu, hit);
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    int at = found + __popc(m & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (hit && at < 8) s_tok[at] = static_cast<int>(i);
    for (int w = 0; w < kFewWarps; ++w) found += s_warp[w];
    __syncthreads();
  }
  __syncthreads();

  // s = A x, split over d_in between the 64 warps of the cluster
  const E* A = static_cast<const E*>(p.a) + static_cast<int64_t>(g) * p.rank * p.d_in;
  const int my_tok = s_tok[row];
  const E* x = my_tok >= 0 ? static_cast<const E*>(p.x) + my_tok * p.x_stride : nullptr;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float acc[MB][4] = {};
  for (int kb = cta * kFewWarps + warp; kb < p.d_in / 32; kb += kCluster * kFewWarps) {
    const int col = kb * 32 + c * 8;
    const uint4 xv = x ? *reinterpret_cast<const uint4*>(x + col) : zero;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int r0 = m * 16 + row, r1 = r0 + 8;
      const uint4 lo = r0 < k ? *reinterpret_cast<const uint4*>(A + static_cast<int64_t>(r0) * p.d_in + col) : zero;
      const uint4 hi = r1 < k ? *reinterpret_cast<const uint4*>(A + static_cast<int64_t>(r1) * p.d_in + col) : zero;
      mma16816<E>(acc[m], lo.x, hi.x, lo.y, hi.y, xv.x, xv.y);
      mma16816<E>(acc[m], lo.z, hi.z, lo.w, hi.w, xv.z, xv.w);
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    float* o = part + (warp * kR + m * 16 + row) * 8 + c * 2;
    *reinterpret_cast<float2*>(o) = make_float2(acc[m][0], acc[m][1]);
    *reinterpret_cast<float2*>(o + 64) = make_float2(acc[m][2], acc[m][3]);
  }
  __syncthreads();
  for (int i = tid; i < kR * 8; i += kFewThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) s += part[w * kR * 8 + i];
    mine[i] = s;
  }
  sm100::cluster_sync();
  // every CTA sums the eight CTAs' parts, in their order
  const float sc = p.scale ? p.scale[g] : 1.0f;
  float* total = part;                                     // [kR][8], the warps' parts are done with
  const uint32_t base = sm100::smem_u32(mine);
  for (int i = tid; i < kR * 8; i += kFewThreads) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) s += ld_cluster(sm100::mapa_shared(base + i * 4, r));
    total[i] = s * sc;
  }
  __syncthreads();
  if (std::is_same<E, __half>::value) {
    // (one warp for each token: the largest magnitude of its s)
    float top = 0.0f;
    for (int r = lane; r < kR; r += 32) top = fmaxf(top, fabsf(total[r * 8 + warp]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float down, up;
    fp16_scaling(top, &down, &up);
    for (int r = lane; r < kR; r += 32) total[r * 8 + warp] *= down;
    if (lane == 0) s_up[warp] = up;
    __syncthreads();
  }
  for (int i = tid; i < kR * 8; i += kFewThreads) {
    E v[kT];
    split<E>(total[i], v);
#pragma unroll
    for (int q = 0; q < kT; ++q) terms[(q * 8 + (i & 7)) * kRow + (i >> 3)] = v[q];
  }
  __syncthreads();

  // y = y_in + B s, split over d_out
  const E* B = static_cast<const E*>(p.b) + static_cast<int64_t>(g) * p.d_out * p.rank;
  const int blocks = (p.d_out + 15) / 16;
  for (int nb = cta * kFewWarps + warp; nb < blocks; nb += kCluster * kFewWarps) {
    const int n0 = nb * 16 + row, n1 = n0 + 8;
    float o[4] = {};
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int col = m * 16 + c * 4;
      if (m * 16 >= k) break;
      uint2 lo = make_uint2(0, 0), hi = lo;
      if (col < k) {
        lo = *reinterpret_cast<const uint2*>(B + static_cast<int64_t>(n0) * p.rank + col);
        if (n1 < p.d_out) hi = *reinterpret_cast<const uint2*>(B + static_cast<int64_t>(n1) * p.rank + col);
      }
      // columns from k on are padding that may hold anything
      lo.x = keep_below(lo.x, col, k); lo.y = keep_below(lo.y, col + 2, k);
      hi.x = keep_below(hi.x, col, k); hi.y = keep_below(hi.y, col + 2, k);
#pragma unroll
      for (int q = 0; q < kT; ++q) {
        const uint2 s = *reinterpret_cast<const uint2*>(terms + (q * 8 + row) * kRow + col);
        mma16816<E>(o, lo.x, hi.x, lo.y, hi.y, s.x, s.y);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = j < 2 ? n0 : n1, slot = c * 2 + (j & 1), tok = s_tok[slot];
      if (tok < 0 || n >= p.d_out) continue;
      float v = o[j];
      if (std::is_same<E, __half>::value) v *= s_up[slot];
      if (p.y_in) v += p.y_in[tok * p.y_in_stride + n];
      p.y[tok * p.y_stride + n] = v;
    }
  }
  sm100::cluster_sync();                                   // no CTA leaves while another may read its sums
}

template <typename E, int MB>
int launch_few(const LoraArgs& p, cudaStream_t st) {
  constexpr int kR = MB * 16;
  constexpr int smem = kFewWarps * kR * 8 * 4 + kR * 8 * 4 + Split<E>::kTerms * 8 * (kR + 8) * 2;
  auto kern = lora_few_kernel<E, MB>;
  if (smem > 48 * 1024 - 256) {
    static std::atomic<uint64_t> done{0};
    if (set_smem_once(kern, smem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tokens * kCluster));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return WUSH_ERR_CUDA;
  return launch_status();
}

template <typename E>
int run_lora(const LoraArgs& p, cudaStream_t st) {
  if (p.rank <= 16) return launch_few<E, 1>(p, st);
  if (p.rank <= 32) return launch_few<E, 2>(p, st);
  if (p.rank <= 64) return launch_few<E, 4>(p, st);
  if (p.rank <= 128) return launch_few<E, 8>(p, st);
  return launch_few<E, 16>(p, st);
}

}  // namespace
}  // namespace wush

using namespace wush;

extern "C" size_t wush_lora_workspace_bytes(int64_t tokens, int64_t d_in, int64_t d_out, int64_t n_adapters,
                                            int64_t rank) {
  (void)d_in; (void)d_out; (void)n_adapters; (void)rank; (void)tokens;
  return 0;
}

extern "C" int wush_lora_add(const wush_lora_args* args, void* stream) {
  if (!args) return WUSH_ERR_INVALID_ARG;
  const wush_lora_args& q = *args;
  if (q.tokens < 0 || q.d_in <= 0 || q.d_in % 32 || q.d_out <= 0 || q.d_out % 8 || q.n_adapters <= 0 || q.rank <= 0 ||
      q.rank % 8)
    return WUSH_ERR_INVALID_ARG;
  if (q.dtype != WUSH_BF16 && q.dtype != WUSH_FP16) return WUSH_ERR_UNSUPPORTED;
  if (q.rank > kMaxRank || q.n_adapters > kMaxAdapters || q.d_in > kMaxWidth || q.d_out > kMaxWidth ||
      q.tokens > kMaxTokens)
    return WUSH_ERR_UNSUPPORTED;
  if (q.tokens == 0) return WUSH_OK;
  if (!q.x || !q.adapter || !q.a || !q.b || !q.y) return WUSH_ERR_INVALID_ARG;
  for (const void* p : {q.x, q.a, q.b, static_cast<const void*>(q.y), static_cast<const void*>(q.y_in)})
    if (!aligned16(p)) return WUSH_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(q.adapter), static_cast<const void*>(q.ranks),
                        static_cast<const void*>(q.scale)})
    if (reinterpret_cast<uintptr_t>(p) & 3) return WUSH_ERR_INVALID_ARG;
  if (q.x_stride < q.d_in || q.x_stride % 8 || q.y_stride < q.d_out || q.y_stride % 4) return WUSH_ERR_INVALID_ARG;
  if (q.y_in && (q.y_in_stride < q.d_out || q.y_in_stride % 4)) return WUSH_ERR_INVALID_ARG;
  const int64_t far = (int64_t(1) << 60) / q.tokens;
  if (q.x_stride > far || q.y_stride > far || (q.y_in && q.y_in_stride > far)) return WUSH_ERR_UNSUPPORTED;
  const Span out = span(q.y, WUSH_FP32, q.y_stride, q.d_out);
  if (overlap(out, span(q.x, q.dtype, q.x_stride, q.d_in), q.tokens)) return WUSH_ERR_INVALID_ARG;
  if (!(q.y == q.y_in && q.y_stride == q.y_in_stride) &&
      overlap(out, span(q.y_in, WUSH_FP32, q.y_in_stride, q.d_out), q.tokens))
    return WUSH_ERR_INVALID_ARG;
  LoraArgs p = {q.x, q.adapter, q.a, q.b, q.ranks, q.scale, q.y_in, q.y, q.x_stride, q.y_in_stride, q.y_stride,
                q.tokens, static_cast<int>(q.d_in), static_cast<int>(q.d_out), static_cast<int>(q.n_adapters),
                static_cast<int>(q.rank)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return q.dtype == WUSH_FP16 ? run_lora<__half>(p, st) : run_lora<__nv_bfloat16>(p, st);
}
