// embed_kernels.cu -- rows of an embedding table, scaled, and the table's gradient from the positions
// sorted by token.
//
//   Y[t] = scale W[tokens[t]]            dW[v] = scale sum over t with tokens[t] = v of dY[t]
//
// The gradient in three launches. First the positions are sorted by token, stably, by one cluster of
// CTAs (a radix sort by digits of at most 9 bits; whole numbers, so the order is always the same), while
// the other SMs write zeros to the table's rows that no token names. Then blocks of kept length of the
// sorted positions are summed, whatever the runs of equal tokens in them are: a frequent token is many
// blocks' work. A run inside a block goes to its row of the table, a run that crosses blocks leaves its
// parts in the workspace, and the third launch adds those in the order of the blocks.
// Sums are fp32, in the order of the positions within a block; no atomics on values.
#include <algorithm>

#include "stream_rows.cuh"

namespace p24 {
namespace {

// ---------------------------------------------------------------- lookup
// A CTA: blockDim.x pieces of 8 columns, blockDim.y rows, U of them for a thread.
template <typename Tw, typename To, int U>
__global__ void __launch_bounds__(256) embed_kernel(const p24_embed_args g, bool wv, bool yv) {
  const int d = static_cast<int>(g.d), c = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * U) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (c >= d) return;
  int tok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    tok[u] = t < g.T ? g.tokens[t] : -1;
  }
  Raw8<Tw> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tok[u] >= 0 && tok[u] < g.V) {
      r[u] = load8(static_cast<const Tw*>(g.W) + static_cast<int64_t>(tok[u]) * g.ldw, c, d, wv);
    } else {
#pragma unroll
      for (unsigned i = 0; i < sizeof(Tw) / 2; ++i) r[u].q[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    if (t >= g.T) break;
    float v[8];
    unpack8(r[u], v);
    const bool in = tok[u] >= 0 && tok[u] < g.V;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = in ? v[k] * g.scale : 0.f;  // a scale of infinity times a 0 that is not there
    store8(static_cast<To*>(g.Y) + t * g.ldy, c, d, yv, v);
  }
}

// ---------------------------------------------------------------- sort
constexpr int kSortThreads = 1024, kSortWarps = 32, kDigit = 9, kBins = 1 << kDigit;
constexpr int kSortCtas = 8;          // the portable cluster size
constexpr int kFillRows = 1 << 17;    // rows of the table that a CTA looks at together: a bit each

struct SortShared {
  uint32_t count[kSortWarps][kBins];  // a warp's elements with each digit; then where its next one goes
  uint32_t total[kBins];              // the CTA's
  uint32_t scan[kSortWarps];
};

__device__ __forceinline__ void cluster_barrier_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t load_cta(const uint32_t* p, int rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// (token, position), by token; a token outside 0..V-1 is V. `ctas`: those that sort, one cluster.
__device__ __forceinline__ void sort_tokens(const int32_t* tokens, int64_t T, int64_t V, int bits, int passes, int2* a, int2* b,
                                            int rank, int ctas, SortShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t warps = static_cast<int64_t>(ctas) * kSortWarps;
  const int64_t span = (T + warps * 32 - 1) / (warps * 32) * 32;
  const int64_t lo = (static_cast<int64_t>(rank) * kSortWarps + warp) * span, hi = min(T, lo + span);
  const int bins = 1 << bits;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    // the last pass writes to a
    const int2* from = ((passes - pass) & 1) ? b : a;
    int2* to = ((passes - pass) & 1) ? a : b;
    auto key_of = [&](int64_t i) {
      if (pass) return __ldcg(from + i);
      const int32_t v = tokens[i];
      return make_int2(v >= 0 && v < V ? v : static_cast<int>(V), static_cast<int>(i));
    };
    for (int i = lane; i < bins; i += 32) sh.count[warp][i] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const int digit = i < hi ? (key_of(i).x >> shift) & (bins - 1) : -1;
      const unsigned peers = __match_any_sync(~0u, digit);
      if (digit >= 0 && lane == __ffs(peers) - 1) sh.count[warp][digit] += __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    uint32_t mine = 0;
    if (tid < bins) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = sh.count[w][tid];
        sh.count[w][tid] = mine;
        mine += n;
      }
      sh.total[tid] = mine;
    }
    uint32_t before = 0, all = mine;
    if (ctas > 1) {
      cluster_barrier_all();
      all = 0;
      if (tid < bins)
        for (int r = 0; r < ctas; ++r) {
          const uint32_t n = load_cta(&sh.total[tid], r);
          if (r < rank) before += n;
          all += n;
        }
    }
    // exclusive sums over the digits
    uint32_t up = all;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const uint32_t n = __shfl_up_sync(~0u, up, i);
      if (lane >= i) up += n;
    }
    if (lane == 31) sh.scan[warp] = up;
    __syncthreads();
    uint32_t base = up - all + before;
    for (int w = 0; w < warp; ++w) base += sh.scan[w];
    if (tid < bins)
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) sh.count[w][tid] += base;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      int2 e = make_int2(0, 0);
      if (i < hi) e = key_of(i);
      const int digit = i < hi ? (e.x >> shift) & (bins - 1) : -1;
      const unsigned peers = __match_any_sync(~0u, digit);
      const uint32_t at = digit >= 0 ? sh.count[warp][digit] : 0;
      __syncwarp();
      if (digit >= 0) {
        if (lane == __ffs(peers) - 1) sh.count[warp][digit] = at + __popc(peers);
        to[at + __popc(peers & ((1u << lane) - 1))] = e;
      }
      __syncwarp();
    }
    // the others' elements are there, and their totals read, before the next pass
    if (ctas > 1) cluster_barrier_all();
    else __syncthreads();
  }
}

// `n` bytes of zeros, by a warp.
__device__ __forceinline__ void zero_row(uint8_t* p, int64_t n, int unit) {
  const int lane = threadIdx.x & 31;
  const int64_t head = min(n, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u));
  const int64_t vecs = (n - head) >> 4, tail = head + (vecs << 4);
  const int64_t ends = (head + n - tail) / unit;
  if (lane < ends) {
    const int64_t at = lane * unit < head ? lane * unit : tail + lane * unit - head;
    if (unit == 2) *reinterpret_cast<uint16_t*>(p + at) = 0;
    else *reinterpret_cast<uint32_t*>(p + at) = 0;
  }
  uint4* q = reinterpret_cast<uint4*>(p + head);
#pragma unroll 4
  for (int64_t i = lane; i < vecs; i += 32) q[i] = make_uint4(0, 0, 0, 0);
}

// CTAs [0, ctas): the sort. The others: zeros for the table's rows without a token.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const p24_embed_bwd_args g, int bits, int passes, int ctas, int2* a, int2* b) {
  extern __shared__ __align__(16) uint8_t raw[];
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) < ctas) {
    sort_tokens(g.tokens, g.T, g.V, bits, passes, a, b, blockIdx.x, ctas, *reinterpret_cast<SortShared*>(raw));
    return;
  }
  uint32_t* used = reinterpret_cast<uint32_t*>(raw);
  const int64_t fills = gridDim.x - ctas, f = blockIdx.x - ctas;
  const int64_t end = g.V * (f + 1) / fills;
  const int unit = g.dw_dtype == P24_BF16 ? 2 : 4;
  for (int64_t lo = g.V * f / fills; lo < end; lo += kFillRows) {
    const int rows = static_cast<int>(min(end - lo, static_cast<int64_t>(kFillRows)));
    __syncthreads();
    for (int i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) used[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < g.T; t += kSortThreads) {
      const int64_t v = g.tokens[t] - lo;
      if (v >= 0 && v < rows) atomicOr(&used[v >> 5], 1u << (v & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < rows; i += kSortWarps)
      if (!(used[i >> 5] >> (i & 31) & 1))
        zero_row(static_cast<uint8_t*>(g.dW) + (lo + i) * g.lddw * unit, g.d * unit, unit);
  }
}

// ---------------------------------------------------------------- sums
constexpr int kBlockMost = 64;  // sorted positions of a block, at most

struct SumArgs {
  p24_embed_bwd_args g;
  const int2* sorted;
  float* parts;  // [blocks, 2, dpad]: a block's part of the run that enters it, and of the one that leaves it
  int64_t dpad;
  int length;    // of a block
  bool dyv, dwv;
};

template <typename To>
__device__ __forceinline__ void put_row(const p24_embed_bwd_args& g, int v, int c, int d, bool vec, float (&s)[8]) {
  To* to = static_cast<To*>(g.dW) + static_cast<int64_t>(v) * g.lddw;
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] *= g.scale;
  if (g.accumulate) {
    float old[8];
    unpack8(load8(static_cast<const To*>(to), c, d, vec), old);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] += old[k];
  }
  store8(to, c, d, vec, s);
}

template <typename Td, typename To, int U>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a) {
  __shared__ int2 e[kBlockMost + 2];  // the block's, with its neighbours around it
  const p24_embed_bwd_args& g = a.g;
  const int d = static_cast<int>(g.d), V = static_cast<int>(g.V);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.length;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.length), g.T - p0));
  const int c = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const int64_t p = p0 + i - 1;
    e[i] = p >= 0 && p < g.T ? a.sorted[p] : make_int2(-1, -1);
  }
  __syncthreads();
  if (c >= d) return;
  const Td* dy = static_cast<const Td*>(g.dY);
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.f;
  int start = 1;
  for (int i0 = 1; i0 <= n; i0 += U) {
    Raw8<Td> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u <= n && e[i0 + u].x < V) r[u] = load8(dy + static_cast<int64_t>(e[i0 + u].y) * g.lddy, c, d, a.dyv);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i > n || e[i].x >= V) break;
      float v[8];
      unpack8(r[u], v);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += v[k];
      if (i < n && e[i + 1].x == e[i].x) continue;
      // a run ends, or the block does
      const bool enters = start == 1 && e[0].x == e[1].x, leaves = i == n && e[n + 1].x == e[n].x;
      if (!enters && !leaves) {
        put_row<To>(g, e[i].x, c, d, a.dwv, s);
      } else {
        float* to = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + (enters ? 0 : 1)) * a.dpad + c;
        reinterpret_cast<float4*>(to)[0] = make_float4(s[0], s[1], s[2], s[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(s[4], s[5], s[6], s[7]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = 0.f;
      start = i + 1;
    }
  }
}

// For each run that crosses blocks, at the first border that it crosses: its parts.
template <typename To>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs a) {
  const p24_embed_bwd_args& g = a.g;
  const int d = static_cast<int>(g.d);
  const int64_t blocks = (g.T + a.length - 1) / a.length;
  const int c = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
  pdl_wait();
  pdl_trigger();
  if (c >= d) return;
  for (int64_t b = blockIdx.x; b + 1 < blocks; b += gridDim.x) {
    const int64_t end = (b + 1) * a.length;
    const int v = a.sorted[end - 1].x;
    if (v >= g.V || a.sorted[end].x != v) continue;
    if (b > 0 && a.sorted[end - a.length].x == v && a.sorted[end - a.length - 1].x == v) continue;  // it came from before
    const float* p = a.parts + (2 * b + 1) * a.dpad + c;
    float s[8];
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w, s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
    // how far it goes: blocks whose first position has the token
    int64_t last = b + 1;
    while (last + 1 < blocks && a.sorted[(last + 1) * a.length].x == v) ++last;
#pragma unroll 4
    for (int64_t q = b + 1; q <= last; ++q) {
      const float* part = a.parts + 2 * q * a.dpad + c;
      const float4 u = reinterpret_cast<const float4*>(part)[0], w = reinterpret_cast<const float4*>(part)[1];
      s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w, s[4] += w.x, s[5] += w.y, s[6] += w.z, s[7] += w.w;
    }
    put_row<To>(g, v, c, d, a.dwv, s);
  }
}

// Sorted positions of a block: as many as leave 8 CTAs for each SM.
int block_length(int64_t T, int64_t d) {
  const int64_t chunks = (d + 1023) / 1024, want = T * chunks / (8 * sm_count());
  int n = 4;
  while (n < kBlockMost && n < want) n *= 2;
  return n;
}
int64_t pad8(int64_t d) { return (d + 7) / 8 * 8; }
int64_t sort_bytes(int64_t T) { return (T * 8 + 255) / 256 * 256; }

dim3 piece_block(int64_t d, int most) {
  const int64_t n = (d + 7) / 8;
  int x = 32;
  while (x < most && x < n) x *= 2;
  return dim3(x);
}

template <typename Td, typename To>
cudaError_t launch_sums(const SumArgs& a, cudaStream_t s) {
  const dim3 block = piece_block(a.g.d, 128);
  const int64_t blocks = (a.g.T + a.length - 1) / a.length;
  const unsigned chunks = static_cast<unsigned>(((a.g.d + 7) / 8 + block.x - 1) / block.x);
  cudaError_t e = launch_pdl(embed_sum_kernel<Td, To, 4>, dim3(static_cast<unsigned>(blocks), chunks), block, 0, s, a);
  if (e != cudaSuccess) return e;
  count_launch();
  if (blocks == 1) return e;
  e = launch_pdl(embed_join_kernel<To>, dim3(static_cast<unsigned>(std::min<int64_t>(blocks - 1, 65535)), chunks), block, 0, s, a);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename Tw, typename To>
cudaError_t launch_embed_as(const p24_embed_args& g, cudaStream_t s) {
  const bool wv = rows_aligned(g.W, g.ldw, g.w_dtype), yv = rows_aligned(g.Y, g.ldy, g.y_dtype);
  dim3 block = piece_block(g.d, 256);
  block.y = 256 / block.x;
  const int64_t n = (g.d + 7) / 8;
  const unsigned chunks = static_cast<unsigned>((n + block.x - 1) / block.x);
  auto go = [&](auto kern, int u) {
    const int64_t rows = static_cast<int64_t>(u) * block.y;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>((g.T + rows - 1) / rows), chunks), block, 0, s, g, wv, yv);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (g.T * n >= 256 * 8 * 4 * sm_count()) return go(embed_kernel<Tw, To, 4>, 4);
  return go(embed_kernel<Tw, To, 1>, 1);
}

}  // namespace

size_t embed_bwd_workspace(int64_t T, int64_t d) {
  const int64_t blocks = (T + block_length(T, d) - 1) / block_length(T, d);
  return static_cast<size_t>(2 * sort_bytes(T) + 2 * blocks * pad8(d) * sizeof(float));
}

cudaError_t launch_embed(const p24_embed_args& g, cudaStream_t s) {
  if (g.w_dtype == P24_BF16) return g.y_dtype == P24_BF16 ? launch_embed_as<bf16, bf16>(g, s) : launch_embed_as<bf16, float>(g, s);
  return g.y_dtype == P24_BF16 ? launch_embed_as<float, bf16>(g, s) : launch_embed_as<float, float>(g, s);
}

cudaError_t launch_embed_bwd(const p24_embed_bwd_args& g, void* ws, cudaStream_t s) {
  SumArgs a{g, nullptr, nullptr, pad8(g.d), block_length(g.T, g.d), rows_aligned(g.dY, g.lddy, g.dy_dtype),
            rows_aligned(g.dW, g.lddw, g.dw_dtype)};
  int2* first = static_cast<int2*>(ws);
  int2* second = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + sort_bytes(g.T));
  a.sorted = first;
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * sort_bytes(g.T));
  int total = 1;  // of the keys 0..V
  while (g.V >> total) ++total;
  const int passes = (total + kDigit - 1) / kDigit, bits = (total + passes - 1) / passes;
  const int ctas = g.T <= 4096 ? 1 : kSortCtas;
  const void* kern = reinterpret_cast<const void*>(embed_sort_kernel);
  int slots = 0;
  cudaError_t e = row_kernel_slots(kern, kSortThreads, ctas, sizeof(SortShared), &slots);
  if (e != cudaSuccess) return e;
  // one cluster sorts; the others, as many as fit, write zeros
  const int64_t grid = (g.accumulate ? 1 : std::max<int64_t>(2, slots)) * ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sizeof(SortShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, g, bits, passes, ctas, first, second);
  if (e != cudaSuccess) return e;
  count_launch();
  if (g.T == 0) return cudaSuccess;
  if (g.dy_dtype == P24_BF16) return g.dw_dtype == P24_BF16 ? launch_sums<bf16, bf16>(a, s) : launch_sums<bf16, float>(a, s);
  return g.dw_dtype == P24_BF16 ? launch_sums<float, bf16>(a, s) : launch_sums<float, float>(a, s);
}

}  // namespace p24
