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
constexpr int kMaxSmem = 227 * 1024;
constexpr int kPlanThreads = 1024, kPlanAdapters = 12288;  // adapters whose counts fit the plan's shared memory
constexpr int kShrinkThreads = 256, kExpandThreads = 256;

struct Work {                                              // in the caller's workspace
  int* n_tiles;
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
  o.n_tiles = reinterpret_cast<int*>(take(16));
  o.tiles = reinterpret_cast<int4*>(take(sizeof(int4) * max_tiles(tokens, n)));
  o.token = reinterpret_cast<int*>(take(4 * tokens));
  o.up = reinterpret_cast<float*>(take(4 * tokens));
  o.terms = take(static_cast<size_t>(tokens) * 3 * row * 2);
  o.row_elems = static_cast<int>(row);
  if (w) *w = o;
  return at;
}

// Exclusive prefix sum over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  const int before = warp ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

// One CTA.  Shared memory: a counter for each adapter and one for the tokens without.
// (The order of an adapter's tokens is left to the atomics.  A token's result is the same
// in every place of a tile: rows of an MMA do not meet, and everything else is per row.)
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const int32_t* __restrict__ adapter, int64_t tokens,
                                                                 int n, int rank, const int32_t* __restrict__ ranks,
                                                                 Work w) {
  extern __shared__ int count[];                           // [n + 1], then the next free slot of each
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i <= n; i += kPlanThreads) count[i] = 0;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  __syncthreads();
  // the adapters of eight tokens of each thread at a time, all asked for before any is used
  int mine8[8];
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + j * kPlanThreads + tid;
      const int g = t < tokens ? adapter[t] : n;
      mine8[j] = t >= tokens ? -1 : g >= 0 && g < n ? g : n;
    }
  };
  for (int64_t t0 = 0; t0 < tokens; t0 += 8 * kPlanThreads) {
    fetch(t0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (t0 + j * kPlanThreads >= tokens) break;
      const int g = mine8[j];
      const uint32_t same = __match_any_sync(0xffffffffu, g);
      if (g >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[g], __popc(same));
    }
  }
  __syncthreads();
  int slots = 0, tiles = 0;
  for (int i0 = 0; i0 <= n; i0 += kPlanThreads) {
    const int i = i0 + tid, c = i <= n ? count[i] : 0, cut = (c + kTile - 1) / kTile;
    int all_c, all_t;
    const int first = slots + block_scan(c, warp_sums, &all_c);
    const int tile = tiles + block_scan(cut, warp_sums, &all_t);
    if (c) {
      int k = 0;
      if (i < n) {
        k = ranks ? ranks[i] : rank;
        k = k < 0 ? 0 : k > rank ? rank : k;
      }
      for (int j = 0; j < cut; ++j)
        w.tiles[tile + j] = make_int4(i, first + j * kTile, c - j * kTile < kTile ? c - j * kTile : kTile, k);
    }
    if (i <= n) count[i] = first;
    slots += all_c;
    tiles += all_t;
  }
  if (tid == 0) *w.n_tiles = tiles;
  __syncthreads();
  for (int64_t t0 = 0; t0 < tokens; t0 += 8 * kPlanThreads) {
    if (tokens > 8 * kPlanThreads) fetch(t0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (t0 + j * kPlanThreads >= tokens) break;
      const int g = mine8[j];
      const uint32_t same = __match_any_sync(0xffffffffu, g);
      const int leader = __ffs(same) - 1;
      int at = 0;
      if (g >= 0 && lane == leader) at = atomicAdd(&count[g], __popc(same));
      at = __shfl_sync(0xffffffffu, at, leader);
      if (g >= 0) w.token[at + __popc(same & ((1u << lane) - 1))] = static_cast<int>(t0 + j * kPlanThreads + tid);
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // the rest of the 16 is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

constexpr int kBk = 64;

// NB: blocks of 8 ranks.  A stage holds 64 columns of the tile's x and of A, rows of 128
// bytes whose 16-byte units are permuted by the row (unit ^ row % 8), so that the MMA
// fragments load without bank conflicts.  Behind the stages: the CTA's s, fp32
// [kTile][kRow], into which the MMA accumulators are added every 1024 columns.  Of a
// stage's four MMA steps the first four warps (16 tokens each) take two and the last four
// the others, so no chain of MMAs is longer than 32 steps.
template <int NB>
__host__ __device__ constexpr int shrink_stages() { return NB <= 4 ? 4 : 3; }
template <int NB>
constexpr int shrink_smem() {
  return shrink_stages<NB>() * (kTile + NB * 8) * 128 + kTile * (NB * 8 + 4) * 4;
}

template <typename E, int NB>
__global__ void __launch_bounds__(kShrinkThreads, NB <= 8 ? 3 : 1) lora_shrink_kernel(const __grid_constant__ LoraArgs p,
                                                                     const __grid_constant__ Work w) {
  constexpr int kR = NB * 8, kRow = kR + 4, kT = Split<E>::kTerms, kStage = (kTile + kR) * 128;
  constexpr int kShrinkStages = shrink_stages<NB>();
  extern __shared__ __align__(128) unsigned char smem[];
  float* sum = reinterpret_cast<float*>(smem + kShrinkStages * kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t splits;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(splits));
  const uint32_t cta = sm100::cluster_ctarank();
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int item = blockIdx.x / splits;
  if (item >= *w.n_tiles) return;
  const int4 tile = w.tiles[item];
  const int k = tile.w, count = tile.z;
  if (k == 0) return;                                      // (all CTAs of a cluster decide alike)
  const E* A = static_cast<const E*>(p.a) + static_cast<int64_t>(tile.x) * p.rank * p.d_in;
  // this CTA's columns
  const int steps = (p.d_in + kBk - 1) / kBk, per = (steps + splits - 1) / splits;
  const int first = cta * per < steps ? cta * per : steps, last = first + per < steps ? first + per : steps;

  const uint32_t base = sm100::smem_u32(smem);
  const int unit = tid & 7, row0 = tid >> 3;               // this thread copies unit ``unit`` of rows row0 + 32 j
  const E* x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = row0 + 32 * j;
    x[j] = r < count ? static_cast<const E*>(p.x) + w.token[tile.y + r] * p.x_stride : nullptr;
  }
  auto load = [&](int step) {
    const int col = step * kBk + unit * 8;
    const bool in = col < p.d_in;                          // (d_in is a multiple of 32)
    const uint32_t to = base + (step - first) % kShrinkStages * kStage + ((unit ^ (row0 & 7)) << 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      cp_async16(to + (row0 + 32 * j) * 128, x[j] && in ? x[j] + col : static_cast<const E*>(p.x), x[j] && in ? 16 : 0);
#pragma unroll
    for (int j = 0; j < (NB + 3) / 4; ++j) {
      const int r = row0 + 32 * j;
      if (r >= kR) break;
      const bool ok = in && r < k;
      cp_async16(to + (kTile + r) * 128, ok ? A + static_cast<int64_t>(r) * p.d_in + col : A, ok ? 16 : 0);
    }
  };
  float acc[NB][4] = {};
  const int wm = warp & 3, wk = warp >> 2;                 // 16 tokens; half of a stage's steps
  const bool active = wm * 16 < count;
  const int frow = wm * 16 + (lane >> 2), fcol = (lane & 3) * 2;
  auto flush = [&](bool fresh) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float2* lo = reinterpret_cast<float2*>(sum + frow * kRow + b * 8 + fcol);
      float2* hi = reinterpret_cast<float2*>(sum + (frow + 8) * kRow + b * 8 + fcol);
      if (fresh) {
        *lo = make_float2(acc[b][0], acc[b][1]);
        *hi = make_float2(acc[b][2], acc[b][3]);
      } else {
        const float2 u = *lo, v = *hi;
        *lo = make_float2(u.x + acc[b][0], u.y + acc[b][1]);
        *hi = make_float2(v.x + acc[b][2], v.y + acc[b][3]);
      }
      acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.0f;
    }
  };
  // the first set of warps stores or adds its accumulators, then the second adds its own
  auto flush_all = [&](bool fresh) {
    if (active && wk == 0) flush(fresh);
    __syncthreads();
    if (active && wk == 1) flush(false);
    __syncthreads();
  };
  bool fresh = true;
#pragma unroll
  for (int s = 0; s < kShrinkStages - 1; ++s) {
    if (first + s < last) load(first + s);
    cp_async_commit();
  }
  for (int step = first; step < last; ++step) {
    cp_async_wait<kShrinkStages - 2>();
    __syncthreads();
    if (step + kShrinkStages - 1 < last) load(step + kShrinkStages - 1);
    cp_async_commit();
    if (active) {
      const uint32_t at = base + (step - first) % kShrinkStages * kStage;
      // FULL: every block of 8 ranks is in use, so that the loads need not wait for tests
      auto multiply = [&](auto full) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBk / 32; ++i) {
          const int ks = wk * (kBk / 32) + i;
          uint32_t a[4];
          const int ar = wm * 16 + (lane & 15);
          ldmatrix4(at + ar * 128 + (((2 * ks + (lane >> 4)) ^ (ar & 7)) << 4), a);
#pragma unroll
          for (int b = 0; b < NB; b += 2) {
            if (!full.value && b * 8 >= k) break;
            uint32_t q[4];
            const int br = b * 8 + (lane & 7) + ((lane >> 4) << 3);
            ldmatrix4(at + (kTile + br) * 128 + (((2 * ks + ((lane >> 3) & 1)) ^ (br & 7)) << 4), q);
            mma16816<E>(acc[b], a[0], a[1], a[2], a[3], q[0], q[1]);
            mma16816<E>(acc[b + 1], a[0], a[1], a[2], a[3], q[2], q[3]);
          }
        }
      };
      if (k > (NB - 2) * 8) multiply(std::true_type{});
      else multiply(std::false_type{});
    }
    if ((step - first) % 16 == 15) {
      flush_all(fresh);
      fresh = false;
    }
  }
  flush_all(fresh);
  sm100::cluster_sync();

  // The cluster's CTAs share the tile's rows; a warp sums the parts of a row in their
  // order, scales, and stores the terms.
  const float sc = p.scale ? p.scale[tile.x] : 1.0f;
  const uint32_t sum_at = sm100::smem_u32(sum);
  E* terms = static_cast<E*>(w.terms);
  const int kp = (k + 15) / 16 * 16;
  for (int r = cta + splits * warp; r < count; r += splits * (kShrinkThreads / 32)) {
    float v[(kR + 31) / 32];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < (kR + 31) / 32; ++i) {
      const int c = i * 32 + lane;
      v[i] = 0.0f;
      if (c < kp) {
        for (uint32_t q = 0; q < splits; ++q) v[i] += ld_cluster(sm100::mapa_shared(sum_at + (r * kRow + c) * 4, q));
        v[i] *= sc;
      }
      top = fmaxf(top, fabsf(v[i]));
    }
    float down = 1.0f, up = 1.0f;
    if (std::is_same<E, __half>::value) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      fp16_scaling(top, &down, &up);
      if (lane == 0) w.up[tile.y + r] = up;
    }
#pragma unroll
    for (int i = 0; i < (kR + 31) / 32; ++i) {
      const int c = i * 32 + lane;
      if (c >= kp) continue;
      E t[kT];
      split<E>(v[i] * down, t);
#pragma unroll
      for (int q = 0; q < kT; ++q)
        terms[(static_cast<int64_t>(tile.y + r) * kT + q) * w.row_elems + c] = t[q];
    }
  }
  sm100::cluster_sync();                                   // no CTA leaves while another may read its sums
}

// A CTA takes a tile and a run of blocks of 64 columns.  The tile's terms stay in shared
// memory; B and y_in come through a ring, ahead of the products.  A warp has 16 tokens x 32
// columns.  Column order: of 16 columns, MMA block 0 takes those with bit 1 clear and block
// 1 the others (the rows of B are put into shared memory in that order), so that a thread's
// values of both blocks are four consecutive columns: one 16-byte access of y each.  y_in
// goes into slots that only the thread itself reads.  Rows of B and of the terms are 16
// bytes longer than the ranks, which spreads a fragment's rows over the banks.
// KS: the rank's MMA steps that have an unrolled loop.
template <typename E, int KS>
__global__ void __launch_bounds__(kExpandThreads) lora_expand_kernel(const __grid_constant__ LoraArgs p,
                                                                     const __grid_constant__ Work w, int stages,
                                                                     int most_run) {
  constexpr int kT = Split<E>::kTerms;
  const int row_bytes = w.row_elems * 2 + 16;
  extern __shared__ __align__(128) unsigned char smem[];   // terms [kT][kTile] rows; per stage: y_in slots, B rows
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = warp & 3, wn = warp >> 2, g = lane >> 2, c = lane & 3;
  constexpr int kSlots = kTile * kCols * 4;
  const int stage_bytes = kSlots + kCols * row_bytes;
  const uint32_t s_base = sm100::smem_u32(smem), ring = s_base + kT * kTile * row_bytes;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  // a run of column blocks as long as still gives every CTA a few items
  const int blocks = (p.d_out + kCols - 1) / kCols, n_tiles = *w.n_tiles;
  int run = static_cast<int>(static_cast<int64_t>(n_tiles) * blocks / (4 * gridDim.x));
  run = run < 2 ? 2 : run > most_run ? most_run : run;
  const int runs = (blocks + run - 1) / run;
  const int64_t items = static_cast<int64_t>(n_tiles) * runs;
  const bool in_place = p.y == p.y_in;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int4 tile = w.tiles[item / runs];
    const int first = static_cast<int>(item % runs) * run, last = first + run < blocks ? first + run : blocks;
    const int k = tile.w, count = tile.z;
    if (k == 0 && in_place) continue;
    const int r0 = wm * 16 + g, r1 = r0 + 8;
    const int64_t t0 = r0 < count ? w.token[tile.y + r0] : -1, t1 = r1 < count ? w.token[tile.y + r1] : -1;
    const int units = (k + 15) / 16 * 2;
    const E* B = static_cast<const E*>(p.b) + static_cast<int64_t>(tile.x) * p.d_out * p.rank;
    const E* S = static_cast<const E*>(w.terms) + static_cast<int64_t>(tile.y) * kT * w.row_elems;
    __syncthreads();                                       // the run before is done with shared memory
    for (int i = tid; i < count * kT * units; i += kExpandThreads) {
      const int r = i / units, u = i % units;              // r: slot * kT + term
      cp_async16(s_base + (r % kT * kTile + r / kT) * row_bytes + u * 16, S + static_cast<int64_t>(r) * w.row_elems + u * 8,
                 16);
    }
    auto load = [&](int block) {
      const int n0 = block * kCols;
      const uint32_t to = ring + (block - first) % stages * stage_bytes;
      for (int i = tid; i < kCols * units; i += kExpandThreads) {
        const int n = i / units, u = i % units, col = u * 8;
        int bytes = n0 + n < p.d_out ? (k - col) * 2 : 0;  // columns from k on are padding that may hold anything
        bytes = bytes < 0 ? 0 : bytes > 16 ? 16 : bytes;
        const int at = (n & ~15) | ((n >> 1) & 1) << 3 | ((n >> 2) & 3) << 1 | (n & 1);
        cp_async16(to + kSlots + at * row_bytes + u * 16, bytes ? B + static_cast<int64_t>(n0 + n) * p.rank + col : B,
                   bytes);
      }
      if (p.y_in) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = n0 + wn * 32 + j * 16 + c * 4;
          if (n >= p.d_out) continue;
          if (t0 >= 0) cp_async16(to + ((2 * j) * kExpandThreads + tid) * 16, p.y_in + t0 * p.y_in_stride + n, 16);
          if (t1 >= 0) cp_async16(to + ((2 * j + 1) * kExpandThreads + tid) * 16, p.y_in + t1 * p.y_in_stride + n, 16);
        }
      }
    };
    for (int s = 0; s < stages - 1; ++s) {
      if (first + s < last) load(first + s);
      cp_async_commit();
    }
    float up0 = 1.0f, up1 = 1.0f;
    if (std::is_same<E, __half>::value && k) {
      if (t0 >= 0) up0 = w.up[tile.y + r0];
      if (t1 >= 0) up1 = w.up[tile.y + r1];
    }
    for (int block = first; block < last; ++block) {
      if (stages == 3) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncthreads();
      if (block + stages - 1 < last) load(block + stages - 1);
      cp_async_commit();
      if (wm * 16 >= count) continue;
      const uint32_t at = ring + (block - first) % stages * stage_bytes;
      float acc[4][4] = {};
      auto step = [&](int ks) __attribute__((always_inline)) {
        uint32_t q[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          ldmatrix4(at + kSlots + (wn * 32 + j * 16 + (lane & 7) + ((lane >> 4) << 3)) * row_bytes +
                        (2 * ks + ((lane >> 3) & 1)) * 16, q[j]);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          uint32_t a[4];
          ldmatrix4(s_base + (t * kTile + wm * 16 + (lane & 15)) * row_bytes + (2 * ks + (lane >> 4)) * 16, a);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma16816<E>(acc[2 * j], a[0], a[1], a[2], a[3], q[j][0], q[j][1]);
            mma16816<E>(acc[2 * j + 1], a[0], a[1], a[2], a[3], q[j][2], q[j][3]);
          }
        }
      };
      if (units == 2 * KS) {                               // the pool's whole rank: a loop without tests
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) step(ks);
      } else {
        for (int ks = 0; ks < units / 2; ++ks) step(ks);
      }
      const float4* slots = reinterpret_cast<const float4*>(smem + (at - s_base));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = block * kCols + wn * 32 + j * 16 + c * 4;
        if (n >= p.d_out) continue;
        float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
        if (p.y_in) {
          u = slots[(2 * j) * kExpandThreads + tid];
          v = slots[(2 * j + 1) * kExpandThreads + tid];
        }
        if (t0 >= 0)
          __stcs(reinterpret_cast<float4*>(p.y + t0 * p.y_stride + n),
                 make_float4(fmaf(acc[2 * j][0], up0, u.x), fmaf(acc[2 * j][1], up0, u.y),
                             fmaf(acc[2 * j + 1][0], up0, u.z), fmaf(acc[2 * j + 1][1], up0, u.w)));
        if (t1 >= 0)
          __stcs(reinterpret_cast<float4*>(p.y + t1 * p.y_stride + n),
                 make_float4(fmaf(acc[2 * j][2], up1, v.x), fmaf(acc[2 * j][3], up1, v.y),
                             fmaf(acc[2 * j + 1][2], up1, v.z), fmaf(acc[2 * j + 1][3], up1, v.w)));
      }
    }
  }
}

template <typename E, int NB>
int launch_shrink(const LoraArgs& p, const Work& w, int64_t tiles, int sms, cudaStream_t st) {
  constexpr int smem = shrink_smem<NB>();
  auto kern = lora_shrink_kernel<E, NB>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, smem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  // Split d_in so that the tiles' clusters fill the SMs once, but not below 256 columns a
  // CTA (the number of tiles is known on the device only: the runs' ends are taken as half
  // a tile each).
  constexpr int kFit = 227 * 1024 / (smem + 1024), kCtas = NB > 8 ? 1 : kFit < 3 ? kFit : 3;
  const int64_t likely = (p.tokens + kTile - 1) / kTile + (p.n_adapters < p.tokens ? p.n_adapters : p.tokens) / 2;
  int64_t splits = kCtas * sms / likely;
  if (splits > p.d_in / 256) splits = p.d_in / 256;
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
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
  if (cudaLaunchKernelEx(&cfg, kern, p, w) != cudaSuccess) return WUSH_ERR_CUDA;
  return launch_status();
}

template <typename E, int KS>
int launch_expand(const LoraArgs& p, const Work& w, int64_t tiles, int sms, cudaStream_t st) {
  // three stages of the ring where two CTAs an SM hold them, else two
  const int row_bytes = w.row_elems * 2 + 16, terms = Split<E>::kTerms * kTile * row_bytes;
  const int stage = kTile * kCols * 4 + kCols * row_bytes;
  const int stages = terms + 3 * stage <= 111 * 1024 ? 3 : 2, smem = terms + stages * stage;
  auto kern = lora_expand_kernel<E, KS>;
  static std::atomic<uint64_t> done{0};
  if (set_smem_once(kern, kMaxSmem, done) != WUSH_OK) return WUSH_ERR_CUDA;
  const int fit = 227 * 1024 / (smem + 1024), ctas = fit < 1 ? 1 : fit < 3 ? fit : 3;
  const int64_t blocks = (p.d_out + kCols - 1) / kCols, slots = int64_t(sms) * ctas, items = tiles * ((blocks + 1) / 2);
  return launch_pdl(kern, static_cast<unsigned>(items < slots ? items : slots), kExpandThreads, smem, st, p, w, stages, 16);
}

template <typename E>
int launch_many(const LoraArgs& p, const Work& w, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return WUSH_ERR_CUDA;
  const int64_t tiles = max_tiles(p.tokens, p.n_adapters);
  const int plan_smem = (p.n_adapters + 1) * 4;
  if (plan_smem > 48 * 1024 - 256) {
    static std::atomic<uint64_t> done{0};
    if (set_smem_once(lora_plan_kernel, (kPlanAdapters + 1) * 4, done) != WUSH_OK) return WUSH_ERR_CUDA;
  }
  int rc = launch_pdl(lora_plan_kernel, 1, kPlanThreads, plan_smem, st, p.adapter, p.tokens, p.n_adapters, p.rank,
                      p.ranks, w);
  if (rc != WUSH_OK) return rc;
  rc = p.rank <= 16    ? launch_shrink<E, 2>(p, w, tiles, sms, st)
       : p.rank <= 32  ? launch_shrink<E, 4>(p, w, tiles, sms, st)
       : p.rank <= 64  ? launch_shrink<E, 8>(p, w, tiles, sms, st)
       : p.rank <= 128 ? launch_shrink<E, 16>(p, w, tiles, sms, st)
                       : launch_shrink<E, 32>(p, w, tiles, sms, st);
  if (rc != WUSH_OK) return rc;
  switch (w.row_elems) {
    case 16: return launch_expand<E, 1>(p, w, tiles, sms, st);
    case 32: return launch_expand<E, 2>(p, w, tiles, sms, st);
    case 48: return launch_expand<E, 3>(p, w, tiles, sms, st);
    case 64: return launch_expand<E, 4>(p, w, tiles, sms, st);
    default: return launch_expand<E, 8>(p, w, tiles, sms, st);
  }
}

// Few tokens (or a pool too large to count in shared memory) go through the cluster
// kernel, whose clusters each look through the adapters of all tokens.
constexpr int kFewTokens = 256;

bool few(int64_t tokens, int64_t n) {
  static const int f = getenv("FEW") ? atoi(getenv("FEW")) : kFewTokens;
  return tokens <= f || n > kPlanAdapters; }

template <typename E>
int run_lora(const LoraArgs& p, void* workspace, cudaStream_t st) {
  if (!few(p.tokens, p.n_adapters)) {
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
  return rank <= kMaxRank && n <= kMaxAdapters && d_in <= kMaxWidth && d_out <= kMaxWidth && tokens <= kMaxTokens;
}

}  // namespace
}  // namespace wush

using namespace wush;

extern "C" size_t wush_lora_workspace_bytes(int64_t tokens, int64_t d_in, int64_t d_out, int64_t n_adapters,
                                            int64_t rank) {
  if (!sizes_ok(tokens, d_in, d_out, n_adapters, rank) || !sizes_taken(tokens, d_in, d_out, n_adapters, rank) ||
      few(tokens, n_adapters))
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
  if (q.x_stride > far || q.y_stride > far || (q.y_in && q.y_in_stride > far)) return WUSH_ERR_UNSUPPORTED;
  const Span out = span(q.y, WUSH_FP32, q.y_stride, q.d_out);
  if (overlap(out, span(q.x, q.dtype, q.x_stride, q.d_in), q.tokens)) return WUSH_ERR_INVALID_ARG;
  if (!(q.y == q.y_in && q.y_stride == q.y_in_stride) &&
      overlap(out, span(q.y_in, WUSH_FP32, q.y_in_stride, q.d_out), q.tokens))
    return WUSH_ERR_INVALID_ARG;
  LoraArgs p = {q.x, q.adapter, q.a, q.b, q.ranks, q.scale, q.y_in, q.y, q.x_stride, q.y_in_stride, q.y_stride,
                q.tokens, static_cast<int>(q.d_in), static_cast<int>(q.d_out), static_cast<int>(q.n_adapters),
                static_cast<int>(q.rank)};
  const size_t need = wush_lora_workspace_bytes(q.tokens, q.d_in, q.d_out, q.n_adapters, q.rank);
  if (need) {
    if (!q.workspace || !aligned16(q.workspace)) return WUSH_ERR_INVALID_ARG;
    if (q.workspace_bytes < need) return WUSH_ERR_BUFFER_TOO_SMALL;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return q.dtype == WUSH_FP16 ? run_lora<__half>(p, q.workspace, st) : run_lora<__nv_bfloat16>(p, q.workspace, st);
}
