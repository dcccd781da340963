// Low-rank adapters of many requests beside a shared projection:
//   y[t] = y_in[t] + scale[g] * B_g (A_g x[t]),   g = adapter[t].
//
// Tokens of one adapter are taken together, so that its matrices are read once for
// up to eight of them (few tokens) or 64 (many).
//
// Precision.  The products of 16-bit inputs are exact in fp32 and s = A x is kept in
// fp32; for the second product s is split into 16-bit terms, so that what rounds is the
// fp32 accumulation:
//   bf16: three bf16 terms, each what the ones before it leave cut to 8 bits: all 24 bits
//         of s, and no finite s becomes an infinity;
//   fp16: two fp16 terms (11 bits each) after a power-of-two scaling of the token's s to
//         below 1, undone exactly on the result.  The second term is held times 2^24 and
//         has a sum of its own, since beside the first it would lie in fp16's subnormals
//         for all but the largest s: 23 bits of an s down to 2^-14 of the token's largest,
//         12 bits at 2^-25 and on to 2^-38.
#include <type_traits>

#include "rowops.cuh"
#include "sm100.cuh"

namespace wush {

static __device__ int g_lora_error = 0;

int read_and_clear_lora_error(int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_lora_error, sizeof(int));
  if (e != cudaSuccess) return e;
  if (*word) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_lora_error, &zero, sizeof(int));
  }
  return e;
}

namespace {

constexpr int64_t kDefaultPolls = int64_t(1) << 40;        // waits end on the timer
constexpr uint64_t kDeadlineNs = 4000000000ull;

// A wait gave up: mark it, and let what is in flight land before the CTA's memory goes.
__device__ __forceinline__ void report_timeout() {
  atomicOr(&g_lora_error, kErrTimeoutBarrier);
  const uint64_t until = sm100::globaltimer_ns() + 200000ull;
  while (sm100::globaltimer_ns() < until) __nanosleep(1000);
}

constexpr int kMaxRank = 256;
constexpr int64_t kMaxAdapters = 1 << 20, kMaxWidth = 1 << 24, kMaxTokens = 1 << 24;
constexpr int64_t kMaxStride = int64_t(1) << 38;           // of a tensor map's rows

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
  int64_t polls;                                           // see kDefaultPolls
  bool mute;                                               // test hook: shrink and expand ask for no operands
};

template <typename E>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<E, __half>::value)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename E>
struct Split;
// The tensor core's additions cut off low bits of the larger operand's, so where terms share a sum the low
// ones go first: of the 48 steps that 256 ranks take, the 32 of bf16's second and third term then work on
// sums of 2^-7 of the result's size, and 16 on the whole.
template <>
struct Split<__nv_bfloat16> {
  static constexpr int kTerms = 3, kSums = 1;              // kSums: sums that the terms' products go to
};
template <>
struct Split<__half> {
  static constexpr int kTerms = 2, kSums = 2;
};
constexpr float kUpSecond = 16777216.0f, kDownSecond = 1.0f / kUpSecond;  // of fp16's second term

// The 16-bit terms of v.  (An infinity is its own first term and leaves nothing.)
template <typename E>
__device__ __forceinline__ void split(float v, E (&t)[Split<E>::kTerms]) {
#pragma unroll
  for (int i = 0; i < Split<E>::kTerms; ++i) {
    if constexpr (std::is_same<E, __half>::value) {
      t[i] = __float2half_rn(v);
      const float got = __half2float(t[i]);
      v = v == got ? 0.0f : (v - got) * kUpSecond;
    } else {
      t[i] = __float2bfloat16_rz(v);
      const float got = __bfloat162float(t[i]);
      v = v == got ? 0.0f : v - got;
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

// |v| for fp16_scaling's ``top``: the largest finite magnitude.
__device__ __forceinline__ float finite_magnitude(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }

__device__ __forceinline__ uint32_t keep_below(uint32_t pair, int col, int k) {   // elements col, col + 1
  return col + 1 < k ? pair : col < k ? pair & 0xffffu : 0u;
}

// ---------------------------------------------------------------------------
// Few tokens: one cluster of eight CTAs takes up to eight tokens of one adapter
// through both products in one launch.  Both run as m16n8k16 MMAs with the adapter's
// matrix as the 16-row operand and the tokens as the 8 columns: the matrices go from
// global memory straight into MMA fragments (the order of k inside a step is free as long
// as both operands share it, so a lane takes 16 consecutive bytes of a row of A, 8 of B).
// ---------------------------------------------------------------------------
constexpr int kCluster = 8, kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kLooks = 2, kLookTokens = kLooks * kFewThreads;      // tokens that the threads of a CTA look at together

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Asks for the 128-byte lines of [p, p + bytes) to be brought into L2, by ``threads`` threads
// of which this is number ``i0``.
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t bytes, int i0, int threads) {
  for (int64_t i = i0 * int64_t(128); i < bytes; i += threads * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + i));
}

__device__ __forceinline__ void st_cluster4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// MB: blocks of 16 ranks held at once.  Shared memory: the warps' partial s
// [8][MB * 16][8], the CTAs' sums [8][MB * 16][8], the terms [kTerms][8][MB * 16 + 8].
//
// What bounds it is latency: of the adapter's number, of A and x, of the cluster's meeting, of B.
// So no load hides behind a branch (what is not there reads something that is): all of a step's
// are in flight before any is used.  B and y_in are on their way into L2 while s is computed, a
// warp asks for several blocks of B (kUnroll) before it multiplies any, and a CTA writes its sums
// to the others before they meet, so that nobody reads across after it.  1 token, 4096 x 4096,
// rank 16: 4.5 us, of which about 0.5 go to the adapter's number, 0.5 to the grouping, 0.6 to A,
// 1.2 to the sums and terms, 0.9 to B and y.  16 tokens, 4096 x 4096, rank 64, one adapter each:
// 9.3 us, 1.9 TB/s; 200 on 48 adapters of rank 32, 4096 x 12288: 22.0 us, 3.3 TB/s.
//
// CTAs an SM.  Three of ranks 17 to 32 have 80 registers a thread and spill some 110 bytes, two of ranks 65
// to 128 spill 68; with one fewer, which do not spill: 200 tokens on 48 adapters, 4096 x 12288, rank 32,
// 28.6 us (22.2 so); 32 tokens on 16, 4096 x 4096, rank 32, 7.3 (8.0); 64 on 64, rank 128, 96.9 (44.1).
constexpr int few_ctas(int mb) { return mb <= 2 ? 3 : mb <= 8 ? 2 : 1; }

template <typename E, int MB>
__global__ void __launch_bounds__(kFewThreads, few_ctas(MB))
    lora_few_kernel(const __grid_constant__ LoraArgs p) {
  constexpr int kR = MB * 16, kT = Split<E>::kTerms, kRow = kR + 8;
  constexpr int kUnroll = MB == 1 ? 4 : MB == 2 ? 3 : MB <= 4 ? 2 : 1, kSteps = MB <= 2 ? 2 : 1;   // blocks of B, steps of A in flight
  extern __shared__ __align__(16) unsigned char smem[];
  float* part = reinterpret_cast<float*>(smem);
  float* parts = part + kFewWarps * kR * 8;                // written by the CTAs of the cluster
  E* terms = reinterpret_cast<E*>(parts + kCluster * kR * 8);
  __shared__ __align__(16) int s_adapter[kLookTokens];
  __shared__ int s_first[kLookTokens], s_tok[8], s_warp[kLooks * kFewWarps], s_before;
  __shared__ float s_up[8];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = lane >> 2, c = lane & 3;
  const int cta = static_cast<int>(sm100::cluster_ctarank());
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  // The tokens of an adapter go in groups of eight in their order (those without an adapter as if
  // they had one of their own).  Up to kLookTokens, a thread looks at one or two tokens and the
  // clusters take the groups in turn; for more, the cluster of a group's first token takes it and
  // the others leave.  (All CTAs of a cluster decide alike.)
  const bool one_look = p.tokens <= kLookTokens;
  int64_t groups = p.tokens;
  int mine[kLooks] = {-2, -2}, before[kLooks] = {};        // the thread's tokens: their adapters, earlier tokens of these
  if (one_look) {
    const int tokens = static_cast<int>(p.tokens);
#pragma unroll
    for (int j = 0; j < kLooks; ++j) {
      if (j * kFewThreads >= tokens) break;
      const int i = j * kFewThreads + tid;
      if (i < tokens) {
        mine[j] = p.adapter[i];
        if (mine[j] < 0 || mine[j] >= p.n_adapters) mine[j] = -1;
      }
      s_adapter[i] = mine[j];
    }
    __syncthreads();
    bool first[kLooks] = {};
#pragma unroll
    for (int j = 0; j < kLooks; ++j) {
      if (j * kFewThreads >= tokens) break;
      const int i0 = j * kFewThreads + warp * 32;          // of the warp's tokens
      if (i0 < tokens) {
#pragma unroll 8
        for (int i = 0; i < i0; i += 4) {
          const int4 q = *reinterpret_cast<const int4*>(s_adapter + i);
          before[j] += (q.x == mine[j]) + (q.y == mine[j]) + (q.z == mine[j]) + (q.w == mine[j]);
        }
        before[j] += __popc(__match_any_sync(0xffffffffu, mine[j]) & ((1u << lane) - 1));
      }
      first[j] = i0 + lane < tokens && before[j] % 8 == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, first[j]);
      if (lane == 0) s_warp[j * kFewWarps + warp] = __popc(m);
    }
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int j = 0; j < kLooks; ++j) {
      if (j * kFewThreads >= tokens) break;
      int at = all + __popc(__ballot_sync(0xffffffffu, first[j]) & ((1u << lane) - 1));
      for (int w = 0; w < kFewWarps; ++w) {
        if (w < warp) at += s_warp[j * kFewWarps + w];
        all += s_warp[j * kFewWarps + w];
      }
      if (first[j]) s_first[at] = j * kFewThreads + tid;
    }
    groups = all;
  }
  for (int64_t group = blockIdx.x / kCluster; group < groups; group += gridDim.x / kCluster) {
  __syncthreads();                                         // the last group's s_tok has been read
  const int64_t t = one_look ? s_first[group] : group;
  int g = one_look ? s_adapter[t] : p.adapter[t];
  if (g < 0 || g >= p.n_adapters) g = -1;
  int k = 0;
  if (g >= 0) {
    k = p.ranks ? p.ranks[g] : p.rank;
    k = k < 0 ? 0 : k > p.rank ? p.rank : k;
  }
  if (k == 0 && p.y == p.y_in) continue;
  if (tid < 8) s_tok[tid] = -1;
  if (one_look) {
#pragma unroll
    for (int j = 0; j < kLooks; ++j)
      if (j * kFewThreads + tid == t) s_before = before[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kLooks; ++j)
      if (mine[j] == g && before[j] >= s_before && before[j] < s_before + 8) s_tok[before[j] - s_before] = j * kFewThreads + tid;
    __syncthreads();
  } else if (k == 0) {                                     // (each such token's own cluster)
    if (tid == 0) s_tok[0] = static_cast<int>(t);
    __syncthreads();
  } else {
    int earlier = 0;
    for (int64_t i0 = 0; i0 < t; i0 += kFewThreads) {
      const int64_t i = i0 + tid;
      earlier += __syncthreads_count(i < t && p.adapter[i] == g);
    }
    if (earlier % 8) return;
    int found = 0;
    for (int64_t i0 = t; i0 < p.tokens && found < 8; i0 += kFewThreads) {
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
  }
  if (k == 0) {                                            // no adapter: y_in passes through, a warp for each token
    if (s_tok[warp] >= 0) {
      const float4* src = reinterpret_cast<const float4*>(p.y_in ? p.y_in + s_tok[warp] * p.y_in_stride : nullptr);
      float4* dst = reinterpret_cast<float4*>(p.y + s_tok[warp] * p.y_stride);
      for (int i0 = cta * 32 + lane; i0 < p.d_out / 4; i0 += kCluster * 32 * 4) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * kCluster * 32;
          v[j] = src ? src[i < p.d_out / 4 ? i : i0] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * kCluster * 32 < p.d_out / 4) dst[i0 + j * kCluster * 32] = v[j];
      }
    }
    continue;
  }
  // this CTA's blocks of 16 columns of y, and their rows of B
  const E* B = static_cast<const E*>(p.b) + static_cast<int64_t>(g) * p.d_out * p.rank;
  const int blocks = (p.d_out + 15) / 16, per = (blocks + kCluster - 1) / kCluster;
  const int nb_first = cta * per < blocks ? cta * per : blocks, nb_last = nb_first + per < blocks ? nb_first + per : blocks;
  const int n_last = nb_last * 16 < p.d_out ? nb_last * 16 : p.d_out;
  // this CTA runs and has read its parts: the others may write to it (nothing is published yet)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  auto prefetch = [&] {                                    // of this CTA's part of B and of y_in into L2
    prefetch_l2(B + static_cast<int64_t>(nb_first) * 16 * p.rank, static_cast<int64_t>(n_last - nb_first * 16) * p.rank * 2,
                tid, kFewThreads);
    if (p.y_in && s_tok[warp] >= 0 && nb_first < nb_last)
      prefetch_l2(p.y_in + s_tok[warp] * p.y_in_stride + nb_first * 16, static_cast<int64_t>(n_last - nb_first * 16) * 4,
                  lane, 32);
  };
  __syncthreads();

  // s = A x, split over d_in between the warps of the cluster
  const E* A = static_cast<const E*>(p.a) + static_cast<int64_t>(g) * p.rank * p.d_in;
  // (Loads take no branch, so that all of a step's are in flight: columns of s without a token read
  // the first one's x, rows from k on read row k - 1; neither is used.)
  const E* x = static_cast<const E*>(p.x) + s_tok[s_tok[row] >= 0 ? row : 0] * p.x_stride;
  float acc[MB][4] = {};
  // (chains of 32 MMAs: see kChain; the warp's part is its lanes' own places)
  auto flush = [&](bool fresh) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      float2* o = reinterpret_cast<float2*>(part + (warp * kR + m * 16 + row) * 8 + c * 2);
      const float2 u = fresh ? make_float2(0.0f, 0.0f) : o[0], v = fresh ? make_float2(0.0f, 0.0f) : o[32];
      o[0] = make_float2(u.x + acc[m][0], u.y + acc[m][1]);
      o[32] = make_float2(v.x + acc[m][2], v.y + acc[m][3]);
      acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
    }
  };
  int steps = 0;
  constexpr int stride = kCluster * kFewWarps;
  for (int kb = cta * kFewWarps + warp; kb < p.d_in / 32; kb += stride * kSteps, steps += kSteps) {
    if (steps && steps % 16 == 0) flush(steps == 16);
    uint4 xv[kSteps], lo[kSteps][MB], hi[kSteps][MB];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int col = (kb + j * stride < p.d_in / 32 ? kb + j * stride : kb) * 32 + c * 8;
      xv[j] = *reinterpret_cast<const uint4*>(x + col);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int r0 = m * 16 + row, r1 = r0 + 8;
        lo[j][m] = *reinterpret_cast<const uint4*>(A + static_cast<int64_t>(r0 < k ? r0 : k - 1) * p.d_in + col);
        hi[j][m] = *reinterpret_cast<const uint4*>(A + static_cast<int64_t>(r1 < k ? r1 : k - 1) * p.d_in + col);
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j == 0 && steps == 0) prefetch();                // (behind the first loads of A, which are needed first)
      if (kb + j * stride >= p.d_in / 32) break;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        mma16816<E>(acc[m], lo[j][m].x, hi[j][m].x, lo[j][m].y, hi[j][m].y, xv[j].x, xv[j].y);
        mma16816<E>(acc[m], lo[j][m].z, hi[j][m].z, lo[j][m].w, hi[j][m].w, xv[j].z, xv[j].w);
      }
    }
  }
  if (steps == 0) prefetch();
  flush(steps <= 16);
  __syncthreads();
  cluster_wait();
  constexpr int kPair = MB == 1 ? 1 : 2;                   // blocks of 16 ranks that a lane loads of B at once
  const int used = (k + kPair * 16 - 1) / (kPair * 16) * (kPair * 16) * 8;    // of s, [rank][token]
  const uint32_t to = sm100::smem_u32(parts + cta * kR * 8);
  for (int i = tid * 4; i < used; i += kFewThreads * 4) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float4 q = *reinterpret_cast<const float4*>(part + w * kR * 8 + i);
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
#pragma unroll
    for (int r = 0; r < kCluster; ++r)
      st_cluster4(sm100::mapa_shared(to + i * 4, r), s);
  }
  cluster_arrive();
  cluster_wait();
  // every CTA sums the CTAs' parts, in their order
  const float sc = p.scale ? p.scale[g] : 1.0f;
  float* total = part;                                     // [kR][8], the warps' parts are done with
  for (int i = tid * 4; i < used; i += kFewThreads * 4) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      const float4 q = *reinterpret_cast<const float4*>(parts + r * kR * 8 + i);
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
    if (i / 8 >= k) s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    *reinterpret_cast<float4*>(total + i) = make_float4(s.x * sc, s.y * sc, s.z * sc, s.w * sc);
  }
  __syncthreads();
  // a warp for each token: its s, scaled (fp16) and split
  {
    float down = 1.0f, up = 1.0f;
    if (std::is_same<E, __half>::value) {
      float top = 0.0f;
      for (int r = lane; r < used / 8; r += 32) top = fmaxf(top, finite_magnitude(total[r * 8 + warp]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      fp16_scaling(top, &down, &up);
      if (lane == 0) s_up[warp] = up;
    }
    for (int r = lane; r < used / 8; r += 32) {
      E v[kT];
      split<E>(total[r * 8 + warp] * down, v);
#pragma unroll
      for (int q = 0; q < kT; ++q) terms[(q * 8 + warp) * kRow + r] = v[q];
    }
  }
  __syncthreads();

  // y = y_in + B s
  const bool is_half = std::is_same<E, __half>::value;
  const int tok0 = s_tok[c * 2], tok1 = s_tok[c * 2 + 1];
  const float up0 = is_half ? s_up[c * 2] : 1.0f, up1 = is_half ? s_up[c * 2 + 1] : 1.0f;
  // (no branches around loads here either: what is beyond this CTA's columns, the adapter's or a
  // group's tokens reads some valid place)
  const float* in0 = p.y_in ? p.y_in + (tok0 >= 0 ? tok0 : s_tok[0]) * p.y_in_stride : nullptr;
  const float* in1 = p.y_in ? p.y_in + (tok1 >= 0 ? tok1 : s_tok[0]) * p.y_in_stride : nullptr;
  float* out0 = tok0 >= 0 ? p.y + tok0 * p.y_stride : nullptr;
  float* out1 = tok1 >= 0 ? p.y + tok1 * p.y_stride : nullptr;
  // A lane's kPair x 8 consecutive bytes of a row of B are the k-places 2 c, 2 c + 1, 2 c + 8 and
  // 2 c + 9 of kPair MMAs; the terms are read in the same order.
  constexpr int kCols8 = kPair * 4;                        // columns of them
  using Piece = typename std::conditional<kPair == 2, uint4, uint2>::type;
  auto words = [](const Piece& v, int e, uint32_t* first, uint32_t* second) {
    if constexpr (kPair == 2) {
      *first = e ? v.z : v.x;
      *second = e ? v.w : v.y;
    } else {
      *first = v.x;
      *second = v.y;
    }
  };
  auto term = [&](int m, int q) {
    return *reinterpret_cast<const Piece*>(terms + (q * 8 + row) * kRow + m * kPair * 16 + c * kCols8);
  };
  constexpr int kM = MB / kPair;
  constexpr bool kHeld = MB <= 4;                          // the terms stay in registers
  Piece held[kHeld ? kM : 1][kT];
  if constexpr (kHeld) {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int q = 0; q < kT; ++q) held[m][q] = term(m, q);
  }
  for (int nb = nb_first + warp * kUnroll; nb < nb_last; nb += kFewWarps * kUnroll) {
    Piece lo[kUnroll][kM], hi[kUnroll][kM];
    float old[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int n0 = (nb + u) * 16 + row, n1 = n0 + 8, at0 = n0 < n_last ? n0 : n_last - 1, at1 = n1 < n_last ? n1 : n_last - 1;
      const E* b0 = B + static_cast<int64_t>(at0) * p.rank;
      const E* b1 = B + static_cast<int64_t>(at1) * p.rank;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int col = m * kPair * 16 + c * kCols8, from = col < p.rank ? col : 0;
        lo[u][m] = *reinterpret_cast<const Piece*>(b0 + from);
        hi[u][m] = *reinterpret_cast<const Piece*>(b1 + from);
      }
      old[u][0] = old[u][1] = old[u][2] = old[u][3] = 0.0f;
      if (p.y_in) {
        old[u][0] = in0[at0];
        old[u][1] = in1[at0];
        old[u][2] = in0[at1];
        old[u][3] = in1[at1];
      }
    }
    if (k != kR) {                                         // columns from k on are padding that may hold anything
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          uint32_t* l = reinterpret_cast<uint32_t*>(&lo[u][m]);
          uint32_t* h = reinterpret_cast<uint32_t*>(&hi[u][m]);
#pragma unroll
          for (int i = 0; i < kPair * 2; ++i) {
            const int col = m * kPair * 16 + c * kCols8 + i * 2;
            l[i] = keep_below(l[i], col, k);
            h[i] = keep_below(h[i], col, k);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int n0 = (nb + u) * 16 + row, n1 = n0 + 8;
      float o[Split<E>::kSums][4] = {};
      // (the low terms first: see Split)
#pragma unroll
      for (int q = kT - 1; q >= 0; --q) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          if (m * kPair * 16 >= k) break;
          const Piece s = kHeld ? held[kHeld ? m : 0][q] : term(m, q);
#pragma unroll
          for (int e = 0; e < kPair; ++e) {
            uint32_t a0, a1, a2, a3, s0, s1;
            words(lo[u][m], e, &a0, &a2);
            words(hi[u][m], e, &a1, &a3);
            words(s, e, &s0, &s1);
            mma16816<E>(o[q % Split<E>::kSums], a0, a1, a2, a3, s0, s1);
          }
        }
      }
      if (is_half) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[0][j] = fmaf(o[Split<E>::kSums - 1][j], kDownSecond, o[0][j]);
      }
      const bool has0 = n0 < n_last, has1 = n1 < n_last;
      if (out0 && has0) out0[n0] = fmaf(o[0][0], up0, old[u][0]);
      if (out1 && has0) out1[n0] = fmaf(o[0][1], up1, old[u][1]);
      if (out0 && has1) out0[n1] = fmaf(o[0][2], up0, old[u][2]);
      if (out1 && has1) out1[n1] = fmaf(o[0][3], up1, old[u][3]);
    }
  }
  }
}

template <typename E, int MB>
int launch_few(const LoraArgs& p, cudaStream_t st) {
  constexpr int kR = MB * 16;
  constexpr int smem = (kFewWarps + kCluster) * kR * 8 * 4 + Split<E>::kTerms * 8 * (kR + 8) * 2;
  auto kern = lora_few_kernel<E, MB>;
  if (smem > 40 * 1024) {                                  // (and the kernel's own arrays)
    static std::atomic<uint64_t> done{0};
    if (set_smem_once(kern, smem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  // As many clusters as lie on the GPU at once (each within one of its eight GPCs); those of up to
  // kLookTokens tokens go on to further groups.  (200 tokens on 48 adapters, 4096 x 12288, rank
  // 32: 21.4 us; a cluster a token, most of which leave at once: some 5 us more.)
  int64_t clusters = p.tokens;
  if (p.tokens > 16 && p.tokens <= kLookTokens) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return WUSH_ERR_CUDA;
    const int64_t most = sms / 8 * few_ctas(MB) / kCluster * 8;
    if (clusters > most) clusters = most > 0 ? most : 1;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kCluster));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return WUSH_ERR_CUDA;
  return launch_status();
}

// ---------------------------------------------------------------------------
// Many tokens: three launches.
//   plan:   sorts the tokens by adapter and cuts each adapter's run into tiles of up to
//           64 tokens;
//   shrink: s = A x for a tile, d_in split over a cluster's CTAs, summed through
//           distributed shared memory and stored as 16-bit terms;
//   expand: y = y_in + B s for a tile and 128 columns at a time.
// What bounds them: the traffic of x in shrink, of y_in and y in expand.
// ---------------------------------------------------------------------------
constexpr int kTile = 64, kCols = 64;
constexpr int kMaxSmem = 226 * 1024;                      // dynamic; the rest for a kernel's own
constexpr int kPlanThreads = 1024, kPlanAdapters = 57344;  // adapters whose counts fit the plan's shared memory
constexpr int kShrinkThreads = 192;

struct Counts {
  int tiles;
  unsigned next;                                           // pieces that expand's CTAs have drawn
};

struct Work {                                              // in the caller's workspace
  Counts* counts;
  int4* tiles;                                             // adapter, first slot, tokens, rank (0: y_in passes through)
  int* token;                                              // token of each slot (tokens sorted by adapter)
  float* up;                                               // per slot: what undoes the scaling of its terms (fp16)
  void* terms;                                             // [slot][kTerms][row_elems] 16-bit
  int row_elems;                                           // rank rounded up to 16
};

int64_t max_tiles(int64_t tokens, int64_t n) {
  return (tokens + kTile - 1) / kTile + (tokens < n + 1 ? tokens : n + 1);
}

size_t work_layout(int64_t tokens, int64_t n, int64_t rank, char* base, Work* w) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  const int64_t row = (rank + 15) / 16 * 16;
  Work o;
  o.counts = reinterpret_cast<Counts*>(take(sizeof(Counts)));
  o.tiles = reinterpret_cast<int4*>(take(sizeof(int4) * max_tiles(tokens, n)));
  o.token = reinterpret_cast<int*>(take(4 * tokens));
  o.up = reinterpret_cast<float*>(take(4 * tokens));
  o.terms = take(static_cast<size_t>(tokens) * 3 * row * 2);
  o.row_elems = static_cast<int>(row);
  if (w) *w = o;
  return at;
}

// Exclusive prefix sums over the CTA's threads of two packed counters, *total the sums:
// tokens in the upper half, tiles in the lower.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint64_t before = 0, t = warp_sums[lane];                // (every warp scans the warps' sums)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  before = __shfl_sync(0xffffffffu, t, warp ? warp - 1 : 0);
  __syncthreads();
  return (warp ? before : 0) + x - v;
}

// One CTA.  ORDERED: an adapter's tokens keep their order, so that the rows of a request lie
// side by side in a tile and shrink can fetch them in blocks: every warp has a stretch of the
// tokens and counters of its own, in shared memory [32][n + 1], with a row of sums behind them.  Otherwise (pools of more
// than kOrderedAdapters) there is one set of counters, and the order is left to the atomics;
// a token's result is the same in every place of a tile, since rows of an MMA do not meet and
// everything else is per row.
constexpr int kOrderedAdapters = 1024;

template <bool ORDERED>
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const int32_t* __restrict__ adapter, int64_t tokens,
                                                                 int n, int rank, const int32_t* __restrict__ ranks,
                                                                 Work w) {
  extern __shared__ int count[];                           // counts, then the next free slot of each
  __shared__ uint64_t warp_sums[32];
  constexpr int kSets = ORDERED ? 32 : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* mine = count + (ORDERED ? warp * (n + 1) : 0);
  int* start = count + (ORDERED ? 32 * (n + 1) : 0);       // adapters' totals, then their first slots
  for (int i = tid; i < kSets * (n + 1); i += kPlanThreads) count[i] = 0;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  __syncthreads();
  // a warp's stretch, 256 tokens at a time, all asked for before any is used
  const int64_t stretch = (tokens + kPlanThreads - 1) / kPlanThreads * 32, from = warp * stretch;
  const int64_t to = from + stretch < tokens ? from + stretch : tokens;
  int group[8];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + j * 32 + lane;
      const int g = t < to ? adapter[t] : 0;
      group[j] = t >= to ? -1 : g >= 0 && g < n ? g : n;
    }
  };
  auto rank_of = [&](int i) {
    const int k = ranks ? ranks[i] : rank;
    return k < 0 ? 0 : k > rank ? rank : k;
  };
  const int my_rank = tid < n ? rank_of(tid) : 0;
  for (int64_t t0 = from; t0 < to; t0 += 256) {
    fetch(t0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (t0 + j * 32 >= to) break;                        // (the whole warp alike)
      const int g = group[j];
      const uint32_t same = __match_any_sync(0xffffffffu, g);
      if (g >= 0 && lane == __ffs(same) - 1) {
        if (ORDERED) mine[g] += __popc(same);
        else atomicAdd(&mine[g], __popc(same));
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // Each adapter's total and the warps' places within it (ORDERED): a warp for an adapter, a
  // lane for a warp's counter.
  if (ORDERED) {
    for (int i = warp; i <= n; i += 32) {
      const int c = count[lane * (n + 1) + i];
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      count[lane * (n + 1) + i] = x - c;
      if (lane == 31) start[i] = x;
    }
    __syncthreads();
  }
  uint64_t base = 0;
  for (int i0 = 0; i0 <= n; i0 += kPlanThreads) {
    const int i = i0 + tid, c = i <= n ? start[i] : 0;
    const int k = i >= n ? 0 : i0 == 0 ? my_rank : rank_of(i), tiles = (c + kTile - 1) / kTile;
    uint64_t all;
    const uint64_t at = base + block_scan(uint64_t(c) << 32 | uint64_t(tiles), warp_sums, &all);
    const int first = static_cast<int>(at >> 32), tile = static_cast<int>(at);
    base += all;
    // an adapter's tiles: its thread writes a few, its warp many
    auto cut = [&](int to_tile, int g, int slot, int tokens_g, int rank_g, int j) {
      const int left = tokens_g - j * kTile;
      w.tiles[to_tile + j] = make_int4(g, slot + j * kTile, left < kTile ? left : kTile, rank_g);
    };
    if (tiles <= 16)
      for (int j = 0; j < tiles; ++j) cut(tile, i, first, c, k, j);
    for (uint32_t many = __ballot_sync(0xffffffffu, tiles > 16); many; many &= many - 1) {
      const int of = __ffs(many) - 1;
      const int c2 = __shfl_sync(0xffffffffu, c, of), k2 = __shfl_sync(0xffffffffu, k, of);
      const int f2 = __shfl_sync(0xffffffffu, first, of), i2 = __shfl_sync(0xffffffffu, i, of);
      const int t2 = __shfl_sync(0xffffffffu, tile, of), nt = __shfl_sync(0xffffffffu, tiles, of);
      for (int j = lane; j < nt; j += 32) cut(t2, i2, f2, c2, k2, j);
    }
    if (i <= n) start[i] = first;
  }
  if (tid == 0) *w.counts = Counts{static_cast<int>(base), 0u};
  __syncthreads();
  for (int64_t t0 = from; t0 < to; t0 += 256) {
    if (stretch > 256) fetch(t0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (t0 + j * 32 >= to) break;
      const int g = group[j];
      const uint32_t same = __match_any_sync(0xffffffffu, g);
      const int leader = __ffs(same) - 1;
      int at = 0;
      if (g >= 0 && lane == leader) {
        if (ORDERED) {
          at = mine[g];
          mine[g] = at + __popc(same);
          at += start[g];
        } else {
          at = atomicAdd(&mine[g], __popc(same));
        }
      }
      at = __shfl_sync(0xffffffffu, at, leader);
      if (g >= 0) w.token[at + __popc(same & ((1u << lane) - 1))] = static_cast<int>(t0 + j * 32 + lane);
      __syncwarp();
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // the rest of the 16 is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Four rows of a matrix whose tensor map has boxes one row high, side by side in shared
// memory; rows beyond the matrix read as zero.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int col, int4 rows, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w),
      "r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int col, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(sm100::smem_u32(bar))
      : "memory");
}

// 16 rows of B in the order that expand's D wants (b_map): row 8 (the map's fourth axis) and on.
__device__ __forceinline__ void tma_tile_b(uint32_t dst, const CUtensorMap* map, int col, int row8, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %4, %4, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row8), "r"(0), "r"(sm100::smem_u32(bar))
      : "memory");
}

// False for a wait that gives up: it sets the CTA's flag, by which the other roles' waits give up
// too.  The thread then asks for nothing more (its roles' barriers are not through their turns), and
// its warp runs on to the CTA's common barriers, where the error is reported and what is in
// flight lands.
__device__ __forceinline__ bool wait_or_flag(uint64_t* bar, uint32_t parity, const LoraArgs& p, int* abort_flag) {
  if (sm100::mbar_wait_bounded(bar, parity, p.polls, kDeadlineNs, abort_flag)) return true;
  *static_cast<volatile int*>(abort_flag) = 1;
  return false;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// ---- tcgen05, 64 rows a tile (one 16-row slice in each quarter of TMEM's lanes)
template <typename E>
__host__ __device__ constexpr uint32_t idesc_f16_m64(uint32_t n) {        // K-major A and B of E, fp32 D
  const uint32_t type = std::is_same<E, __half>::value ? 0u : 1u;
  return (1u << 4) | (type << 7) | (type << 10) | ((n >> 3) << 17) | ((64u >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(sm100::desc_kmajor_sw128(a)), "l"(sm100::desc_kmajor_sw128(b)), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 lanes x 8 columns: the warp's slice of a 64-row D, held like an m16n8 accumulator
// (lane: row lane / 4 and + 8, columns 2 (lane % 4) and + 1).
__device__ __forceinline__ void tmem_ld_16x8(uint32_t addr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}

constexpr int kBk = 128;                                  // columns of d_in a stage: two operand tiles of 64

// One warp asks for the tiles of x (rows gathered by TMA) and of A, one issues the MMAs, four
// take D out of TMEM.  A stage holds 128 columns as two halves of 64, rows of 128 bytes with
// the 128-byte swizzle.  D is added to fp32 registers and begun anew every kChain stages: the
// tensor core's own additions cut off low bits, and 32 of them in a row stay near fp32's
// rounding of the sums (4096 tokens x 12288, rank 128: 5.7e-7 relative to the result; with
// the second product's low terms last, when both were measured, 1.0e-6, and 2.8e-6 with a chain over a CTA's whole d_in).
//
// What bounds it: 4096 tokens x 12288, rank 64, read 113 MB from DRAM and 277 MB from L2 (A
// once a tile) in some 31 us, the tensor pipe active for a quarter of it.
constexpr int kChain = 4;

template <int R>
struct Shrink {
  static constexpr int kHalf = (kTile + R) * 128, kStage = 2 * kHalf;
  static constexpr int kStages = R <= 128 ? 3 : 2;
  static constexpr int kAcc = R <= 128 ? 2 : 1;            // D's that chains take in turn
  static constexpr int kTmem = kAcc * R < 32 ? 32 : kAcc * R;
  static constexpr int kRow = R + 4;                       // floats of a row of the CTA's s, laid over the stages
  static constexpr int kSmem = kStages * kStage + 1024;    // (the swizzle's 8-row groups are 1024-byte aligned)
  static constexpr int kCtas = 227 * 1024 / (kSmem + 1536);   // an SM
  static_assert(kTile * kRow * 4 <= kStages * kStage, "s fits over the stages");
  // CTAs of a cluster wait for one another, so none may hold an SM's place while it waits for
  // TMEM that a CTA in the same state holds.  A kernel's share of TMEM is no larger than its
  // share of shared memory: whatever CTAs an SM holds, their TMEM is there.
  static_assert(kTmem * 227 <= 512 * (kSmem / 1024), "TMEM goes by shared memory");
};

template <typename E, int R>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const __grid_constant__ LoraArgs p,
                                                                     const __grid_constant__ Work w,
                                                                     const __grid_constant__ CUtensorMap map_x,
                                                                     const __grid_constant__ CUtensorMap map_x8,
                                                                     const __grid_constant__ CUtensorMap map_a) {
  using L = Shrink<R>;
  constexpr int kT = Split<E>::kTerms;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[L::kStages], empty[L::kStages], d_full[L::kAcc], d_empty[L::kAcc];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const uint32_t base = (sm100::smem_u32(smem_raw) + 1023u) & ~1023u;
  float* sum = reinterpret_cast<float*>(smem_raw + (base - sm100::smem_u32(smem_raw)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t splits;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(splits));
  const uint32_t cta = sm100::cluster_ctarank();
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < L::kStages; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < L::kAcc; ++i) {
      sm100::mbar_init(&d_full[i], 1);
      sm100::mbar_init(&d_empty[i], 4);
    }
    sm100::fence_barrier_init();
    sm100::prefetch_tmap(&map_x);
    sm100::prefetch_tmap(&map_x8);
    sm100::prefetch_tmap(&map_a);
  }
  __syncwarp();
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int item = blockIdx.x / splits;
  if (item >= w.counts->tiles) return;
  const int4 tile = w.tiles[item];
  const int k = tile.w, count = tile.z;
  if (k == 0) return;                                      // (all CTAs of a cluster decide alike)
  if (warp == 0) sm100::tmem_alloc(&tmem_slot, L::kTmem);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // this CTA's columns
  const int steps = (p.d_in + kBk - 1) / kBk, per = (steps + splits - 1) / splits;
  const int first = cta * per < steps ? cta * per : steps, n = (first + per < steps ? first + per : steps) - first;
  const uint32_t ranks16 = (k + 15) / 16 * 16;             // columns of D that the MMAs compute
  float total[R / 8][4] = {};
  if (warp == 4) {
    // lane: half of the stage, eight rows of x: one block where they follow one another
    // (4096 tokens x 12288, rank 64: 31.6 us, 40.7 us with all rows gathered), else two gathers (rows without a token
    // lie beyond x and read as zero; groups without one are left as they are)
    const int half = (lane >> 3) & 1, row = (lane & 7) * 8, none = static_cast<int>(p.tokens);
    const int groups = (count + 7) / 8;
    const bool mine = lane < 16 && row < count;
    int rows[8];
    bool block = row + 8 <= count;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      rows[j] = mine && row + j < count ? w.token[tile.y + row + j] : none;
      block = block && rows[j] == rows[0] + j;
    }
    bool live = !p.mute;
    for (int i = 0; i < n; ++i) {
      const int s = i % L::kStages, col = (first + i) * kBk;
      live = live && wait_or_flag(&empty[s], ((i / L::kStages) & 1) ^ 1, p, &abort_flag);
      const uint32_t to = base + s * L::kStage;
      if (lane == 0 && live) {
        sm100::mbar_arrive_expect_tx(&full[s], 2 * (R + groups * 8) * 128);
        tma_tile(to + kTile * 128, &map_a, col, tile.x * p.rank, &full[s]);
        tma_tile(to + L::kHalf + kTile * 128, &map_a, col + 64, tile.x * p.rank, &full[s]);
      }
      __syncwarp();
      const uint32_t dst = to + half * L::kHalf + row * 128;
      if (mine && block && live) {
        tma_tile(dst, &map_x8, col + half * 64, rows[0], &full[s]);
      } else if (mine && live) {
        tma_gather4(dst, &map_x, col + half * 64, make_int4(rows[0], rows[1], rows[2], rows[3]), &full[s]);
        tma_gather4(dst + 512, &map_x, col + half * 64, make_int4(rows[4], rows[5], rows[6], rows[7]), &full[s]);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f16_m64<E>(ranks16);
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages, chain = i / kChain, d = chain % L::kAcc;
        if (i % kChain == 0 && !wait_or_flag(&d_empty[d], ((chain / L::kAcc) & 1) ^ 1, p, &abort_flag)) break;
        if (!wait_or_flag(&full[s], (i / L::kStages) & 1, p, &abort_flag)) break;
        sm100::tc_fence_after();
        const uint32_t at = base + s * L::kStage;
#pragma unroll
        for (int ks = 0; ks < kBk / 16; ++ks) {
          const uint32_t a = at + (ks >> 2) * L::kHalf + (ks & 3) * 32;
          tc_mma(tmem + d * R, a, a + kTile * 128, idesc, i % kChain != 0 || ks > 0);
        }
        sm100::tc_commit(&empty[s]);
        if (i % kChain == kChain - 1 || i == n - 1) sm100::tc_commit(&d_full[d]);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    bool live = true;
    for (int chain = 0; chain * kChain < n; ++chain) {
      const int d = chain % L::kAcc;
      live = live && wait_or_flag(&d_full[d], (chain / L::kAcc) & 1, p, &abort_flag);
      sm100::tc_fence_after();
#pragma unroll
      for (int b = 0; b < R / 8; b += 4) {                 // (four loads in flight)
        float v[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (b + q < R / 8)
            tmem_ld_16x8(tmem + (static_cast<uint32_t>(warp * 32) << 16) + d * R + (b + q) * 8, v[q]);
        sm100::tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (b + q < R / 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) total[b + q][e] += v[q][e];
          }
      }
      sm100::tc_fence_before();
      if (lane == 0) sm100::mbar_arrive(&d_empty[d]);
    }
  }
  __syncthreads();                                         // the stages have been read: s goes over them
  if (tid == 0 && *static_cast<volatile int*>(&abort_flag)) report_timeout();
  if (warp < 4) {
#pragma unroll
    for (int b = 0; b < R / 8; ++b) {                      // (columns from ranks16 on are never read)
      float* o = sum + (warp * 16 + (lane >> 2)) * L::kRow + b * 8 + (lane & 3) * 2;
      *reinterpret_cast<float2*>(o) = make_float2(total[b][0], total[b][1]);
      *reinterpret_cast<float2*>(o + 8 * L::kRow) = make_float2(total[b][2], total[b][3]);
    }
  }
  sm100::tc_fence_before();
  sm100::cluster_sync();
  if (warp == 0) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, L::kTmem);
  }

  // The cluster's CTAs share the tile's rows; a warp sums the parts of a row in their
  // order, scales, and stores the terms.  (Ranks from k on are padding: A may hold anything
  // there.)
  const float sc = p.scale ? p.scale[tile.x] : 1.0f;
  const uint32_t sum_at = sm100::smem_u32(sum);
  E* terms = static_cast<E*>(w.terms);
  for (int r = cta + splits * warp; r < count; r += splits * (kShrinkThreads / 32)) {
    float v[(R + 31) / 32];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < (R + 31) / 32; ++i) {
      const int c = i * 32 + lane;
      v[i] = 0.0f;
      if (c < k) {
        float part[8];
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          part[q] = q < splits ? ld_cluster(sm100::mapa_shared(sum_at + (r * L::kRow + c) * 4, q)) : 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[i] += part[q];
        v[i] *= sc;
      }
      top = fmaxf(top, finite_magnitude(v[i]));
    }
    float down = 1.0f, up = 1.0f;
    if (std::is_same<E, __half>::value) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      fp16_scaling(top, &down, &up);
      if (lane == 0) w.up[tile.y + r] = up;
    }
#pragma unroll
    for (int i = 0; i < (R + 31) / 32; ++i) {
      const int c = i * 32 + lane;
      if (c >= static_cast<int>(ranks16)) continue;
      E t[kT];
      split<E>(v[i] * down, t);
#pragma unroll
      for (int q = 0; q < kT; ++q)
        terms[(static_cast<int64_t>(tile.y + r) * kT + q) * w.row_elems + c] = t[q];
    }
  }
  sm100::cluster_sync();                                   // no CTA leaves while another may read its sums
}

// A CTA goes along a tile in blocks of 64 columns: D = B s is one 64 x 64 product in TMEM.
//
// The terms lie side by side in k, term t of rank j at k = t * row_elems + j, in operand tiles
// of 64 (128-byte rows, 128-byte swizzle); each term's steps meet the same rows of B.  D comes
// back in the layout of an m16n8 accumulator; of 16 columns, its block 0 is given those with
// bit 1 clear and block 1 the others (TMA brings B's rows in that order), so that a thread's
// values of both blocks are four consecutive columns: one 16-byte access of y each.
//
// One warp asks for the terms and B, one issues the MMAs, one draws pieces of work, eight add D
// to y_in and store.  These fetch their own y_in, by asynchronous copies into slots that only the
// thread itself reads, so the roles meet on barriers in shared memory alone.
//
// What bounds it: y_in and y, which pass once.  8192 tokens x 17408, rank 16: 1.11 GB of DRAM
// traffic in 203 us, 5.5 TB/s.
constexpr int kExpandThreads = 352;
constexpr int kAddThreads = 256;

struct Expand {
  int b_bytes, terms_bytes, b_slots, y_slots, smem;
};

template <typename E>
Expand expand_layout(int row_elems) {
  Expand l;
  l.terms_bytes = (Split<E>::kTerms * row_elems + 63) / 64 * kTile * 128;
  l.b_bytes = (row_elems + 63) / 64 * kCols * 128;
  // two CTAs an SM where they fit, with up to four slots of y_in and of B; else one
  const int y = kTile * kCols * 4, half = 111 * 1024, room = l.terms_bytes + 2 * (y + l.b_bytes) <= half ? half : kMaxSmem - 1024;
  l.b_slots = l.y_slots = 2;
  int left = room - l.terms_bytes - 2 * (y + l.b_bytes);
  for (int i = 0; i < 2; ++i) {
    if (left >= l.b_bytes) ++l.b_slots, left -= l.b_bytes;
    if (left >= y) ++l.y_slots, left -= y;
  }
  l.smem = l.terms_bytes + l.b_slots * l.b_bytes + l.y_slots * y + 1024;
  // (a CTA's share of TMEM, 256 columns of 512 for fp16, is no larger than its share of shared
  // memory: see Shrink)
  if (l.smem < 112 * 1024 && Split<E>::kSums > 1) l.smem = 112 * 1024;
  return l;
}

template <typename E>
__global__ void __launch_bounds__(kExpandThreads, 2) lora_expand_kernel(const __grid_constant__ LoraArgs p,
                                                                     const __grid_constant__ Work w,
                                                                     const __grid_constant__ Expand l,
                                                                     const __grid_constant__ CUtensorMap map_s,
                                                                     const __grid_constant__ CUtensorMap map_b) {
  constexpr int kT = Split<E>::kTerms, kSums = Split<E>::kSums, kSlot = kTile * kCols * 4;
  constexpr int kD = kSums * kCols;                        // columns of TMEM that one D takes, of two in turn
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t b_full[4], b_empty[4], d_full[2], d_empty[2], s_full, s_empty, piece_full[2],
      piece_empty[2];
  __shared__ unsigned piece[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const uint32_t s_base = (sm100::smem_u32(smem_raw) + 1023u) & ~1023u, b_ring = s_base + l.terms_bytes;
  const uint32_t y_ring = b_ring + l.b_slots * l.b_bytes;
  unsigned char* smem = smem_raw + (s_base - sm100::smem_u32(smem_raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      sm100::mbar_init(&b_full[i], 1);
      sm100::mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&d_full[i], 1);
      sm100::mbar_init(&d_empty[i], kAddThreads / 32);
      sm100::mbar_init(&piece_full[i], 1);
      sm100::mbar_init(&piece_empty[i], kAddThreads / 32 + 2);
    }
    sm100::mbar_init(&s_full, 1);
    sm100::mbar_init(&s_empty, 1);
    sm100::fence_barrier_init();
    sm100::prefetch_tmap(&map_s);
    sm100::prefetch_tmap(&map_b);
  }
  __syncwarp();
  if (warp == 8) sm100::tmem_alloc(&tmem_slot, 2 * kD);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  // All tiles' column blocks lie in one row, cut into pieces that the CTAs take as they come to
  // them: the first piece by the CTA's number, the later ones from a counter (SMs do not all get
  // the same share of the memory's bandwidth).  The first warp draws a piece ahead of its use
  // and passes it to the roles.
  const int blocks = (p.d_out + kCols - 1) / kCols;
  const int64_t all = static_cast<int64_t>(w.counts->tiles) * blocks;
  // (A short row goes in equal pieces: a tile's terms are fetched anew for each piece.)
  const int64_t even = (all + gridDim.x - 1) / gridDim.x;
  const int64_t size = even < 64 ? (even > 0 ? even : 1) : even / 6 < 32 ? even / 6 : 32;
  struct Piece {
    int4 tile;                                             // adapter, first slot, tokens, rank
    int first, blocks;
  };
  int turn = 0;
  struct Slot {                                            // of a ring, and the parity of its turn
    int i;
    uint32_t turn;
    __device__ __forceinline__ void next(int slots) {
      if (++i == slots) i = 0, turn ^= 1;
    }
  };
  // Calls f for each stretch of a piece within one tile, piece after piece, until none is left
  // (or given out: a wait gave up).
  auto for_pieces = [&](auto f) __attribute__((always_inline)) {
    for (;; ++turn) {
      if (!__all_sync(0xffffffffu, wait_or_flag(&piece_full[turn & 1], (turn >> 1) & 1, p, &abort_flag))) return;
      int64_t pos = piece[turn & 1] * size;
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&piece_empty[turn & 1]);
      if (pos >= all) return;
      const int64_t to = pos + size < all ? pos + size : all;
      while (pos < to) {
        Piece q;
        const int64_t tile = all >> 32 ? pos / blocks : static_cast<uint32_t>(pos) / static_cast<uint32_t>(blocks);
        q.tile = w.tiles[tile];
        q.first = static_cast<int>(pos - tile * blocks);
        q.blocks = to - pos < blocks - q.first ? static_cast<int>(to - pos) : blocks - q.first;
        f(q);
        pos += q.blocks;
      }
    }
  };

  if (warp == 10) {
    if (lane == 0) {
      unsigned index = blockIdx.x;
      for (int i = 0;; ++i) {
        if (!wait_or_flag(&piece_empty[i & 1], ((i >> 1) & 1) ^ 1, p, &abort_flag)) break;
        if (*static_cast<volatile int*>(&abort_flag)) break;
        piece[i & 1] = index;
        sm100::mbar_arrive(&piece_full[i & 1]);
        if (index * size >= all) break;
        index = gridDim.x + atomicAdd(&w.counts->next, 1u);
      }
    }
    __syncwarp();
  } else
  if (warp == 8) {
    int ns = 0;                                            // tiles' terms asked for so far
    bool live = !p.mute;
    Slot slot = {0, 1};                                    // of B
    for_pieces([&](const Piece& q) {
      const int k = q.tile.w, units = (k + 63) / 64;
      if (k == 0) return;
      if (!wait_or_flag(&s_empty, (ns & 1) ^ 1, p, &abort_flag)) live = false;
      ++ns;
      if (lane == 0 && live) {
        sm100::mbar_arrive_expect_tx(&s_full, l.terms_bytes);
        for (int i = 0; i < l.terms_bytes / (kTile * 128); ++i)
          tma_tile(s_base + i * (kTile * 128), &map_s, i * 64, q.tile.y, &s_full);
      }
      const int row8 = static_cast<int>(static_cast<int64_t>(q.tile.x) * p.d_out / 8) + q.first * (kCols / 8);
      for (int b = 0; b < q.blocks; ++b, slot.next(l.b_slots)) {
        const int s = slot.i;
        if (!wait_or_flag(&b_empty[s], slot.turn, p, &abort_flag)) live = false;
        if (lane == 0 && live) sm100::mbar_arrive_expect_tx(&b_full[s], units * kCols * 128);
        __syncwarp();
        // (columns beyond d_out read the next adapter's rows; their results are not stored)
        for (int i = live ? lane : units * 4; i < units * 4; i += 32)
          tma_tile_b(b_ring + s * l.b_bytes + (i >> 2) * (kCols * 128) + (i & 3) * 2048, &map_b, (i >> 2) * 64,
                     row8 + b * (kCols / 8) + (i & 3) * 2, &b_full[s]);
      }
    });
  } else if (warp == 9) {
    int nb = 0, ns = 0;
    bool live = true;
    Slot slot = {0, 0};
    constexpr uint32_t idesc = idesc_f16_m64<E>(kCols);
    for_pieces([&](const Piece& q) {
      const int k = q.tile.w, kp = (k + 15) / 16 * 16;
      if (k == 0) return;
      if (!wait_or_flag(&s_full, ns & 1, p, &abort_flag)) live = false;
      ++ns;
      for (int b = 0; b < q.blocks; ++b, ++nb, slot.next(l.b_slots)) {
        const int s = slot.i, d = nb & 1;
        const uint32_t at = b_ring + s * l.b_bytes;
        if (!wait_or_flag(&b_full[s], slot.turn, p, &abort_flag)) live = false;
        if (k < kp) {
          // columns from k on are padding that may hold anything: the last step's become zero
          for (int r = lane; r < kCols; r += 32)
            for (int c = k; c < kp; ++c)
              *reinterpret_cast<uint16_t*>(smem + (at - s_base) + (c >> 6) * (kCols * 128) + r * 128 +
                                           ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2) = 0;
          sm100::fence_proxy_async_smem();
          __syncwarp();
        }
        if (!wait_or_flag(&d_empty[d], ((nb >> 1) & 1) ^ 1, p, &abort_flag)) live = false;
        sm100::tc_fence_after();
        if (lane == 0 && live) {
          for (int i = 0; i < kT; ++i)
            for (int ks = 0; ks < kp; ks += 16) {
              const int t = kSums == 1 ? kT - 1 - i : i;   // (the low terms first: see Split)
              const int pos_k = t * w.row_elems + ks;
              tc_mma(tmem + d * kD + t % kSums * kCols, s_base + (pos_k >> 6) * (kTile * 128) + (pos_k & 63) * 2,
                     at + (ks >> 6) * (kCols * 128) + (ks & 63) * 2, idesc,
                     (i > 0 && kSums == 1) || ks > 0);
            }
          sm100::tc_commit(&b_empty[s]);
          sm100::tc_commit(&d_full[d]);
          if (b == q.blocks - 1) sm100::tc_commit(&s_empty);
        }
        __syncwarp();
      }
    });
  } else {
    const int wm = warp & 3, wn = warp >> 2, g = lane >> 2, c = lane & 3;
    const bool in_place = p.y == p.y_in;
    int nb = 0;
    for_pieces([&](const Piece& q) {
      const int k = q.tile.w, count = q.tile.z;
      if (k == 0 && in_place) return;
      const int r0 = wm * 16 + g, r1 = r0 + 8;
      const int64_t t0 = r0 < count ? w.token[q.tile.y + r0] : -1, t1 = r1 < count ? w.token[q.tile.y + r1] : -1;
      const int col = q.first * kCols + wn * 32 + c * 4;
      const float* src0 = p.y_in ? p.y_in + t0 * p.y_in_stride + col : nullptr;
      const float* src1 = p.y_in ? p.y_in + t1 * p.y_in_stride + col : nullptr;
      float* dst0 = p.y + t0 * p.y_stride + col;
      float* dst1 = p.y + t1 * p.y_stride + col;
      const bool some = wm * 16 < count;                   // of the warp's rows
      int to = 0, from = 0;                                // slots: the next to fill, to read
      auto fetch = [&](int b) {
        if (p.y_in && some && b < q.blocks) {
          const uint32_t slot = y_ring + to * kSlot + tid * 16;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int n = b * kCols + j * 16;
            if (col + n >= p.d_out) continue;
            if (t0 >= 0) cp_async16(slot + 2 * j * kAddThreads * 16, src0 + n, 16);
            if (t1 >= 0) cp_async16(slot + (2 * j + 1) * kAddThreads * 16, src1 + n, 16);
          }
        }
        cp_async_commit();
        to = to + 1 == l.y_slots ? 0 : to + 1;
      };
      float up0 = 1.0f, up1 = 1.0f;
      if (std::is_same<E, __half>::value && k) {
        if (t0 >= 0) up0 = w.up[q.tile.y + r0];
        if (t1 >= 0) up1 = w.up[q.tile.y + r1];
      }
      for (int b = 0; b < l.y_slots - 1; ++b) fetch(b);
      for (int b = 0; b < q.blocks; ++b) {
        fetch(b + l.y_slots - 1);                          // (into the slot that was read last)
        if (l.y_slots == 4) cp_async_wait<3>();
        else if (l.y_slots == 3) cp_async_wait<2>();
        else cp_async_wait<1>();
        float acc[4][4] = {};
        if (k) {
          const int d = nb & 1;
          wait_or_flag(&d_full[d], (nb >> 1) & 1, p, &abort_flag);
          ++nb;
          if (some) {
            sm100::tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tmem_ld_16x8(tmem + (static_cast<uint32_t>(wm * 32) << 16) + d * kD + wn * 32 + j * 8, acc[j]);
            if constexpr (kSums == 2) {
              float low[4][4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tmem_ld_16x8(tmem + (static_cast<uint32_t>(wm * 32) << 16) + d * kD + kCols + wn * 32 + j * 8, low[j]);
              sm100::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(low[j][e], kDownSecond, acc[j][e]);
            } else {
              sm100::tmem_ld_wait();
            }
            sm100::tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&d_empty[d]);
        }
        const float4* slots = reinterpret_cast<const float4*>(smem + (y_ring - s_base) + from * kSlot) + tid;
        from = from + 1 == l.y_slots ? 0 : from + 1;
        if (!some) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = b * kCols + j * 16;
          if (col + n >= p.d_out) continue;
          float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
          if (p.y_in) {
            u = slots[2 * j * kAddThreads];
            v = slots[(2 * j + 1) * kAddThreads];
          }
          if (t0 >= 0)
            __stcs(reinterpret_cast<float4*>(dst0 + n),
                   make_float4(fmaf(acc[2 * j][0], up0, u.x), fmaf(acc[2 * j][1], up0, u.y),
                               fmaf(acc[2 * j + 1][0], up0, u.z), fmaf(acc[2 * j + 1][1], up0, u.w)));
          if (t1 >= 0)
            __stcs(reinterpret_cast<float4*>(dst1 + n),
                   make_float4(fmaf(acc[2 * j][2], up1, v.x), fmaf(acc[2 * j][3], up1, v.y),
                               fmaf(acc[2 * j + 1][2], up1, v.z), fmaf(acc[2 * j + 1][3], up1, v.w)));
        }
      }
    });
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (*static_cast<volatile int*>(&abort_flag)) {          // (the same for all threads: no role waits any more)
    if (tid == 0) report_timeout();
    __syncthreads();
  }
  if (warp == 8) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 2 * kD);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn get_encode() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A 16-bit matrix [rows, cols], in boxes of 64 columns x box_rows with the 128-byte swizzle.
template <typename E>
bool tensor_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
  EncodeFn enc = get_encode();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
  return enc && enc(map, std::is_same<E, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// B's rows [rows, rank] as n = 8 h + 4 c + 2 b + e, axes (column, e, c, h, b), in boxes of 64 columns x
// 16 rows: rows with b = 0 first, so that D's blocks of eight columns hold those with bit 1 clear
// and set in turn.
template <typename E>
bool b_map(CUtensorMap* map, const void* p, int64_t rows, int64_t rank) {
  EncodeFn enc = get_encode();
  const cuuint64_t r = static_cast<cuuint64_t>(rank), dims[5] = {r, 2, 2, static_cast<cuuint64_t>(rows / 8), 2};
  const cuuint64_t strides[4] = {r * 2, r * 8, r * 16, r * 4};
  const cuuint32_t box[5] = {64, 2, 2, 2, 2}, estr[5] = {1, 1, 1, 1, 1};
  return enc && enc(map, std::is_same<E, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    5, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E, int R>
int launch_shrink(const LoraArgs& p, const Work& w, int64_t tiles, int sms, cudaStream_t st) {
  constexpr int smem = Shrink<R>::kSmem;
  auto kern = lora_shrink_kernel<E, R>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, smem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  // Split d_in so that the tiles' clusters fill the SMs once, but not below 256 columns a
  // CTA (the number of tiles is known on the device only: the runs' ends are taken as half
  // a tile each).
  const int64_t likely = (p.tokens + kTile - 1) / kTile + (p.n_adapters < p.tokens ? p.n_adapters : p.tokens) / 2;
  // (A cluster lies within one of the GPU's eight GPCs.)
  const int64_t gpc = sms / 8 * Shrink<R>::kCtas;
  int64_t splits = 8;
  while (splits > 1 && (gpc / splits * 8 < likely || splits > p.d_in / 256)) --splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  CUtensorMap map_x, map_x8, map_a;
  if (!tensor_map<E>(&map_x, p.x, p.tokens, p.d_in, p.x_stride, 1) ||
      !tensor_map<E>(&map_x8, p.x, p.tokens, p.d_in, p.x_stride, 8) ||
      !tensor_map<E>(&map_a, p.a, int64_t(p.n_adapters) * p.rank, p.d_in, p.d_in, R))
    return WUSH_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, kern, p, w, map_x, map_x8, map_a) != cudaSuccess) return WUSH_ERR_CUDA;
  return launch_status();
}

template <typename E>
int launch_expand(const LoraArgs& p, const Work& w, int64_t tiles, int sms, cudaStream_t st) {
  const Expand l = expand_layout<E>(w.row_elems);
  auto kern = lora_expand_kernel<E>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, kMaxSmem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  const int64_t blocks = (p.d_out + kCols - 1) / kCols, items = tiles * blocks;
  const int64_t slots = int64_t(sms) * (l.smem <= kMaxSmem / 2 ? 2 : 1);
  CUtensorMap map_s, map_b;
  if (!tensor_map<E>(&map_s, w.terms, p.tokens, Split<E>::kTerms * w.row_elems, Split<E>::kTerms * w.row_elems, kTile) ||
      !b_map<E>(&map_b, p.b, int64_t(p.n_adapters) * p.d_out, p.rank))
    return WUSH_ERR_CUDA;
  return launch_pdl(kern, static_cast<unsigned>(items < slots ? items : slots), kExpandThreads, l.smem, st, p, w, l, map_s,
                    map_b);
}

template <typename E>
int launch_many(const LoraArgs& p, const Work& w, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return WUSH_ERR_CUDA;
  const int64_t tiles = max_tiles(p.tokens, p.n_adapters);
  const bool ordered = p.n_adapters <= kOrderedAdapters;
  const int plan_smem = (p.n_adapters + 1) * 4 * (ordered ? 33 : 1);
  auto plan = ordered ? lora_plan_kernel<true> : lora_plan_kernel<false>;
  if (plan_smem > 48 * 1024 - 256) {
    static std::atomic<uint64_t> done[2] = {{0}, {0}};
    const int most = ordered ? (kOrderedAdapters + 1) * 33 * 4 : (kPlanAdapters + 1) * 4;
    if (set_smem_once(plan, most, done[ordered]) != WUSH_OK) return WUSH_ERR_CUDA;
  }
  int rc = launch_pdl(plan, 1, kPlanThreads, plan_smem, st, p.adapter, p.tokens, p.n_adapters, p.rank, p.ranks, w);
  if (rc != WUSH_OK) return rc;
  rc = p.rank <= 16    ? launch_shrink<E, 16>(p, w, tiles, sms, st)
       : p.rank <= 32  ? launch_shrink<E, 32>(p, w, tiles, sms, st)
       : p.rank <= 64  ? launch_shrink<E, 64>(p, w, tiles, sms, st)
       : p.rank <= 128 ? launch_shrink<E, 128>(p, w, tiles, sms, st)
                       : launch_shrink<E, 256>(p, w, tiles, sms, st);
  if (rc != WUSH_OK) return rc;
  return launch_expand<E>(p, w, tiles, sms, st);
}

// Few tokens (or a pool too large to count in shared memory, or for a tensor map) go through the
// cluster kernel: up to 256, or up to 512 where the pool may hold an adapter for every eight of
// them.  Measured on both sides, the cluster kernel first: 256 tokens on 48 adapters, 4096 x 12288,
// rank 32: 22.9 and 48.3 us; on 12, 5120 x 4104, rank 48: 21.2 and 18.5; on 4, 12288 x 4096, rank 64:
// 18.2 and 23.1.  512 tokens, 4096 x 4096, on 64 adapters of rank 64: 35.6 and 45.4; on 256 of rank
// 16: 40.3 and 76.2; all on one of 64, rank 64: 36.3 and 20.0; on 4 of 4, 12288 x 4096: 42.9 and 26.5.
constexpr int kFewTokens = 256;

constexpr int64_t kMostFewTokens = 4096;                   // a cluster's look through all tokens stays short

bool large_pool(int64_t n, int64_t d_out) { return n > kPlanAdapters || n * d_out > 0x7fffffff; }
bool few(int64_t tokens, int64_t n, int64_t d_out) {
  return tokens <= kFewTokens || (tokens <= kLookTokens && n >= tokens / 8) || large_pool(n, d_out);
}

template <typename E>
int run_lora(const LoraArgs& p, void* workspace, cudaStream_t st) {
  if (!few(p.tokens, p.n_adapters, p.d_out)) {
    Work w;
    work_layout(p.tokens, p.n_adapters, p.rank, static_cast<char*>(workspace), &w);
    return launch_many<E>(p, w, st);
  }
  if (p.rank <= 16) return launch_few<E, 1>(p, st);
  if (p.rank <= 32) return launch_few<E, 2>(p, st);
  if (p.rank <= 64) return launch_few<E, 4>(p, st);
  if (p.rank <= 128) return launch_few<E, 8>(p, st);
  return launch_few<E, 16>(p, st);
}

bool sizes_ok(int64_t tokens, int64_t d_in, int64_t d_out, int64_t n, int64_t rank) {
  return tokens >= 0 && d_in > 0 && d_in % 32 == 0 && d_out > 0 && d_out % 8 == 0 && n > 0 && rank > 0 && rank % 8 == 0;
}
bool sizes_taken(int64_t tokens, int64_t d_in, int64_t d_out, int64_t n, int64_t rank) {
  return rank <= kMaxRank && n <= kMaxAdapters && d_in <= kMaxWidth && d_out <= kMaxWidth && tokens <= kMaxTokens &&
         (tokens <= kMostFewTokens || !large_pool(n, d_out));
}

}  // namespace
}  // namespace wush

using namespace wush;

extern "C" size_t wush_lora_workspace_bytes(int64_t tokens, int64_t d_in, int64_t d_out, int64_t n_adapters,
                                            int64_t rank) {
  if (!sizes_ok(tokens, d_in, d_out, n_adapters, rank) || !sizes_taken(tokens, d_in, d_out, n_adapters, rank) ||
      few(tokens, n_adapters, d_out))
    return 0;
  return work_layout(tokens, n_adapters, rank, nullptr, nullptr);
}

extern "C" int wush_lora_add(const wush_lora_args* args, void* stream) {
  if (!args) return WUSH_ERR_INVALID_ARG;
  const wush_lora_args& q = *args;
  if (!sizes_ok(q.tokens, q.d_in, q.d_out, q.n_adapters, q.rank)) return WUSH_ERR_INVALID_ARG;
  if (q.dtype != WUSH_BF16 && q.dtype != WUSH_FP16) return WUSH_ERR_UNSUPPORTED;
  if (!sizes_taken(q.tokens, q.d_in, q.d_out, q.n_adapters, q.rank)) return WUSH_ERR_UNSUPPORTED;
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
  if (q.x_stride > far || q.x_stride > kMaxStride || q.y_stride > far || (q.y_in && q.y_in_stride > far))
    return WUSH_ERR_UNSUPPORTED;
  const Span out = span(q.y, WUSH_FP32, q.y_stride, q.d_out);
  if (overlap(out, span(q.x, q.dtype, q.x_stride, q.d_in), q.tokens)) return WUSH_ERR_INVALID_ARG;
  if (!(q.y == q.y_in && q.y_stride == q.y_in_stride) &&
      overlap(out, span(q.y_in, WUSH_FP32, q.y_in_stride, q.d_out), q.tokens))
    return WUSH_ERR_INVALID_ARG;
  LoraArgs p = {q.x, q.adapter, q.a, q.b, q.ranks, q.scale, q.y_in, q.y, q.x_stride, q.y_in_stride, q.y_stride,
                q.tokens, static_cast<int>(q.d_in), static_cast<int>(q.d_out), static_cast<int>(q.n_adapters),
                static_cast<int>(q.rank), g_wait_limit_override > 0 ? g_wait_limit_override : kDefaultPolls,
                g_wait_limit_override > 0};
  const size_t need = wush_lora_workspace_bytes(q.tokens, q.d_in, q.d_out, q.n_adapters, q.rank);
  if (need) {
    if (!q.workspace || !aligned16(q.workspace)) return WUSH_ERR_INVALID_ARG;
    if (q.workspace_bytes < need) return WUSH_ERR_BUFFER_TOO_SMALL;
    const Span ws = {static_cast<const char*>(q.workspace), 0, static_cast<int64_t>(need)};
    for (const Span& t : {out, span(q.x, q.dtype, q.x_stride, q.d_in), span(q.y_in, WUSH_FP32, q.y_in_stride, q.d_out)})
      if (t.p && ws.p < t.p + (q.tokens - 1) * t.stride + t.width && t.p < ws.p + ws.width) return WUSH_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return q.dtype == WUSH_FP16 ? run_lora<__half>(p, q.workspace, st) : run_lora<__nv_bfloat16>(p, q.workspace, st);
}
