// embed_kernels.cu -- rows of an embedding table, scaled, and the table's gradient from the positions
// sorted by token.
//
//   Y[t] = scale W[tokens[t]]            dW[v] = scale sum over t with tokens[t] = v of dY[t]
//
// The gradient in four launches. The positions are sorted by token, stably, by a cluster of eight CTAs (a radix sort by
// digits of at most 9 bits) or, if they are few, by counting; whole numbers, so the order is always the same. A kernel
// beside that writes zeros to the table. Then blocks of kept length of the sorted positions are summed, whatever the runs
// of equal tokens in them are: a frequent token is many blocks' work. A run inside a block goes to its row of the table,
// a run that crosses blocks leaves its parts in the workspace, and the last launch adds those in the order of the blocks.
// Sums are fp32, in the order of the positions within a block; no atomics on values.
//
// Lookups are bound by memory (16384 x 4096 bf16 to fp32 51 us), the gradient by the zeros where the table is large (the
// same over 131072 to fp32 325 us, 6.6 TB/s) and by the sort's dependent passes where it is small or narrow (16384 x 128
// over 5000 25 us, of which the sort is 13).
#include <algorithm>

#include "stream_rows.cuh"

namespace p24 {
namespace {

// Neighbouring columns that are moved at once, where rows are aligned.
template <typename A, typename B>
constexpr int piece() {
  return sizeof(A) == 4 || sizeof(B) == 4 ? 4 : 8;
}

// ---------------------------------------------------------------- lookup
// A CTA: blockDim.x threads with 8 columns each, blockDim.y rows, U of them for a thread.
template <typename Tw, typename To, int U, int E>
__global__ void __launch_bounds__(256) embed_kernel(const p24_embed_args g) {
  const Columns<E> k(blockIdx.y, threadIdx.x, blockDim.x, static_cast<int>(g.d));
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * U) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (k.none()) return;
  int tok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    tok[u] = t < g.T ? g.tokens[t] : -1;
  }
  Loaded<E, Tw> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tok[u] >= 0 && tok[u] < g.V) r[u] = load_columns(static_cast<const Tw*>(g.W) + static_cast<int64_t>(tok[u]) * g.ldw, k);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    if (t >= g.T) break;
    float v[8];
    const bool in = tok[u] >= 0 && tok[u] < g.V;
    if (in) values(r[u], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in ? v[i] * g.scale : 0.f;
    store_columns(static_cast<To*>(g.Y) + t * g.ldy, k, v);
  }
}

// ---------------------------------------------------------------- sort
constexpr int kSortThreads = 1024, kSortWarps = 32, kDigit = 9, kBins = 1 << kDigit;
constexpr int kSortCtas = 8;          // the portable cluster size
constexpr int kHeld = 4;

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

// (token, position), by token; a token outside 0..V-1 is V. By a cluster, through a and b. (16384 tokens over 5000: one CTA
// 46 us, a cluster of 8 14.)
__device__ __forceinline__ void sort_tokens(const int32_t* tokens, int64_t T, int64_t V, int bits, int passes, int2* a, int2* b,
                                            int rank, SortShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t warps = static_cast<int64_t>(kSortCtas) * kSortWarps;
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
    int2 e[kHeld];  // some of a warp's elements, loaded together
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int64_t i = i0 + 32 * u + lane;
        e[u] = i < hi ? key_of(i) : make_int2(-1, 0);
      }
    };
    for (int i = lane; i < bins; i += 32) sh.count[warp][i] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kHeld) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        if (i0 + 32 * u >= hi) break;
        const int digit = e[u].x < 0 ? -1 : (e[u].x >> shift) & (bins - 1);
        const unsigned peers = __match_any_sync(~0u, digit);
        if (digit >= 0 && lane == __ffs(peers) - 1) sh.count[warp][digit] += __popc(peers);
        __syncwarp();
      }
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
    uint32_t before = 0, all = 0;
    cluster_barrier_all();
    if (tid < bins)
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        const uint32_t n = load_cta(&sh.total[tid], r);
        if (r < rank) before += n;
        all += n;
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
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kHeld) {
      if (span > 32 * kHeld) load(i0);  // else they are still here
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        if (i0 + 32 * u >= hi) break;
        const int digit = e[u].x < 0 ? -1 : (e[u].x >> shift) & (bins - 1);
        const unsigned peers = __match_any_sync(~0u, digit);
        const uint32_t at = digit >= 0 ? sh.count[warp][digit] : 0;
        __syncwarp();
        if (digit >= 0) {
          if (lane == __ffs(peers) - 1) sh.count[warp][digit] = at + __popc(peers);
          to[at + __popc(peers & ((1u << lane) - 1))] = e[u];
        }
        __syncwarp();
      }
    }
    // the others' elements are there, and their totals read, before the next pass
    cluster_barrier_all();
  }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const p24_embed_bwd_args g, int bits, int passes, int2* a, int2* b) {
  extern __shared__ __align__(16) uint8_t raw[];
  pdl_wait();
  pdl_trigger();
  sort_tokens(g.tokens, g.T, g.V, bits, passes, a, b, blockIdx.x, *reinterpret_cast<SortShared*>(raw));
}

// The same for fewer tokens, a warp each: an element's place is the number of those before it. (The whole gradient of 300 x
// 1000 bf16 over 2000 6.9 us, by one CTA 10.2; of 1000 x 4 over 131072 8.4 and 15.1; of 4000 x 1000 over 8000 18.1, by a
// cluster 21.0; of 8192 x 1024 over 32000 31.3 and 27.4.)
constexpr int kRankMost = 4096, kRankThreads = 1024;
__device__ __forceinline__ int below(const int4& k, int x) { return (k.x < x) + (k.y < x) + (k.z < x) + (k.w < x); }
__global__ void __launch_bounds__(kRankThreads) embed_rank_kernel(const int32_t* tokens, int T, int V, int2* to) {
  extern __shared__ __align__(16) int keys[];
  const int lane = threadIdx.x & 31, me = blockIdx.x * (kRankThreads / 32) + (threadIdx.x >> 5), chunks = (T + 127) / 128;
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < chunks * 128; i += kRankThreads) {
    const int32_t v = i < T ? tokens[i] : 0x7fffffff;
    keys[i] = i < T ? (v >= 0 && v < V ? v : V) : 0x7fffffff;
  }
  __syncthreads();
  if (me >= T) return;
  const int mine = keys[me], own = me / 128;
  const int4* q = reinterpret_cast<const int4*>(keys) + lane;
  int place = 0;
#pragma unroll 4
  for (int c = 0; c < own; ++c) place += below(q[32 * c], mine + 1);  // equal ones are before it
  const int4 k = q[32 * own];
  const int before = me - (128 * own + 4 * lane);  // of these four
  place += (k.x < mine + (before > 0)) + (k.y < mine + (before > 1)) + (k.z < mine + (before > 2)) + (k.w < mine + (before > 3));
#pragma unroll 4
  for (int c = own + 1; c < chunks; ++c) place += below(q[32 * c], mine);
  place = __reduce_add_sync(~0u, place);
  if (lane == 0) to[place] = make_int2(mine, me);
}

// ---------------------------------------------------------------- zeros
// `n` bytes of zeros by `threads` threads, of which this is the i-th: 16 bytes at a time between boundaries of 128.
__device__ __forceinline__ void zero_bytes(uint8_t* p, int64_t n, int unit, int i, int threads) {
  const int64_t head = min(n, static_cast<int64_t>((128 - (reinterpret_cast<uintptr_t>(p) & 127u)) & 127u));
  const int64_t vecs = (n - head) / 16, tail = head + vecs * 16;
#pragma unroll 4
  for (int64_t k = i; k < vecs; k += threads) reinterpret_cast<uint4*>(p + head)[k] = make_uint4(0, 0, 0, 0);
  for (int64_t e = static_cast<int64_t>(i) * unit; e < head + n - tail; e += threads * unit) {
    uint8_t* at = p + (e < head ? e : tail + e - head);
    if (unit == 2) *reinterpret_cast<uint16_t*>(at) = 0;
    else *reinterpret_cast<uint32_t*>(at) = 0;
  }
}

// A table's zeros, its rows with a token among them: many small CTAs, which the hardware starts in the order of memory.
// (1 GB in 141 us, 7.6 TB/s; by CTAs that stay and take every n-th piece, stores or bulk copies of any size, 157 to 171.
// Zeros for the rows without a token only, from the SMs that do not sort: 16384 x 4096 over 131072, fp32, 371 us, like
// this 325; over 32000 121 and 117; 2000 x 2000 over 8000, bf16, 21.4 and 22.4.) It needs nothing of the sort's that was
// launched before it and does not wait for it: all of the sort's CTAs had waited for what came before them when they let
// this kernel start. But the sums, which wait for this one, need the sort: the last CTA here waits for it at its end.
// `first`: there was no sort.
constexpr int kZeroThreads = 256, kZeroBytes = kZeroThreads * 4 * 16;
struct Zeros {
  uint8_t* p;
  int64_t n;         // bytes, of a row where there are rows
  int64_t rows, ld;  // rows of a table with gaps, bytes from one to the next; or 0
  int each;          // rows of a CTA
  int unit;
  bool first;
};
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(const Zeros z) {
  if (z.first) pdl_wait();
  pdl_trigger();
  if (z.rows == 0) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kZeroBytes - (blockIdx.x ? reinterpret_cast<uintptr_t>(z.p) & 127u : 0);
    const int64_t end = static_cast<int64_t>(blockIdx.x + 1) * kZeroBytes - (reinterpret_cast<uintptr_t>(z.p) & 127u);
    zero_bytes(z.p + at, min(end, z.n) - at, z.unit, threadIdx.x, kZeroThreads);
  } else {
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * z.each, end = min(r0 + z.each, z.rows);
    for (int64_t r = r0 + (threadIdx.x >> 5); r < end; r += kZeroThreads / 32)
      zero_bytes(z.p + r * z.ld, z.n, z.unit, threadIdx.x & 31, 32);
  }
  if (!z.first && blockIdx.x == gridDim.x - 1) pdl_wait();
}

cudaError_t launch_zeros(const p24_embed_bwd_args& g, cudaStream_t s) {
  const int unit = size_of(g.dw_dtype);
  const int64_t bytes = g.d * unit;
  Zeros z{static_cast<uint8_t*>(g.dW), bytes, g.V, g.lddw * unit, static_cast<int>(8 * std::max<int64_t>(1, 2048 / bytes)), unit, g.T == 0};
  int64_t grid = (g.V + z.each - 1) / z.each;
  if (g.lddw == g.d || g.V == 1) {
    z.n = g.V * bytes, z.rows = 0;
    grid = (z.n + (reinterpret_cast<uintptr_t>(z.p) & 127u) + kZeroBytes - 1) / kZeroBytes;
  }
  const cudaError_t e = launch_pdl(embed_zero_kernel, dim3(static_cast<unsigned>(grid)), dim3(kZeroThreads), 0, s, z);
  if (e == cudaSuccess) count_launch();
  return e;
}

// ---------------------------------------------------------------- sums
constexpr int kBlockMost = 64;  // sorted positions of a block, at most
constexpr int kSumThreads = 128, kJoinThreads = 512;

struct SumArgs {
  p24_embed_bwd_args g;
  const int2* sorted;
  float* parts;  // [blocks, 2, wide]: a block's part of the run that enters it, and of the one that leaves it
  int64_t wide;  // 8 for each thread of a row's chunks
  int length;    // of a block
};

// A thread's 8 sums among the parts.
__device__ __forceinline__ float* part_of(const SumArgs& a, int64_t block, int which, int width) {
  return a.parts + (2 * block + which) * a.wide + (static_cast<int64_t>(blockIdx.y) * width + threadIdx.x) * 8;
}

template <int E, typename To>
__device__ __forceinline__ void put_row(const p24_embed_bwd_args& g, int v, const Columns<E>& k, float (&s)[8]) {
  To* to = static_cast<To*>(g.dW) + static_cast<int64_t>(v) * g.lddw;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] *= g.scale;
  if (g.accumulate) {
    float old[8];
    values(load_columns(static_cast<const To*>(to), k), old);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += old[i];
  }
  store_columns(to, k, s);
}

template <typename Td, typename To, int U, int E>
__global__ void __launch_bounds__(kSumThreads, E == 1 ? 4 : sizeof(Td) == 4 ? 7 : 8) embed_sum_kernel(const SumArgs a) {
  __shared__ int2 e[kBlockMost + 2];  // the block's, with its neighbours around it
  const p24_embed_bwd_args& g = a.g;
  const int V = static_cast<int>(g.V);
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.length;
  const int n = static_cast<int>(min(static_cast<int64_t>(a.length), g.T - p0));
  const Columns<E> k(blockIdx.y, threadIdx.x, blockDim.x, static_cast<int>(g.d));
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const int64_t p = p0 + i - 1;
    e[i] = p >= 0 && p < g.T ? a.sorted[p] : make_int2(-1, -1);
  }
  __syncthreads();
  if (k.none()) return;
  const Td* dy = static_cast<const Td*>(g.dY);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
  int start = 1;
  for (int i0 = 1; i0 <= n && e[i0].x < V; i0 += U) {
    Loaded<E, Td> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u <= n && e[i0 + u].x < V) r[u] = load_columns(dy + static_cast<int64_t>(e[i0 + u].y) * g.lddy, k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i > n || e[i].x >= V) break;
      float v[8];
      values(r[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += v[j];
      if (i < n && e[i + 1].x == e[i].x) continue;
      // a run ends, or the block does
      const bool enters = start == 1 && e[0].x == e[1].x, leaves = i == n && e[n + 1].x == e[n].x;
      if (!enters && !leaves) {
        put_row<E, To>(g, e[i].x, k, s);
      } else {
        float* to = part_of(a, blockIdx.x, enters ? 0 : 1, blockDim.x);
        reinterpret_cast<float4*>(to)[0] = make_float4(s[0], s[1], s[2], s[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(s[4], s[5], s[6], s[7]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = 0.f;
      start = i + 1;
    }
  }
}

// For each run that crosses blocks, at the first border that it crosses: its parts, added up by blockDim.y groups of
// threads that take neighbouring ones, and then group by group.
template <typename To, int E>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const SumArgs a) {
  __shared__ float groups[kJoinThreads][8];
  const p24_embed_bwd_args& g = a.g;
  const int64_t blocks = (g.T + a.length - 1) / a.length;
  const Columns<E> k(blockIdx.y, threadIdx.x, blockDim.x, static_cast<int>(g.d));
  const int me = threadIdx.y * blockDim.x + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  for (int64_t b = blockIdx.x; b + 1 < blocks; b += gridDim.x) {
    const int64_t end = (b + 1) * a.length;
    const int v = a.sorted[end - 1].x, next = a.sorted[end].x;
    const int first = a.sorted[end - a.length].x, before = b > 0 ? a.sorted[end - a.length - 1].x : -1;
    if (v >= g.V || next != v || (first == v && before == v)) continue;  // no run crosses, or it came from before
    // the blocks whose first position has the token
    int64_t n = 0;
    for (;;) {
      const int64_t q = b + 1 + n + me;
      const int more = __syncthreads_count(q < blocks && a.sorted[q * a.length].x == v);
      n += more;
      if (more < static_cast<int>(blockDim.x * blockDim.y)) break;
    }
    const int64_t each = (n + 1 + blockDim.y - 1) / blockDim.y;  // with the part that leaves block b, which is the first
    const int64_t lo = threadIdx.y * each, hi = min(n + 1, lo + each);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll 8
    for (int64_t q = lo; q < hi; ++q) {
      const float* p = part_of(a, b + q, q == 0 ? 1 : 0, blockDim.x);
      const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
      s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w, s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) groups[me][i] = s[i];
    __syncthreads();
    if (threadIdx.y == 0 && !k.none()) {
      for (int y = 1; y < static_cast<int>(blockDim.y); ++y)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += groups[y * blockDim.x + threadIdx.x][i];
      put_row<E, To>(g, v, k, s);
    }
    __syncthreads();
  }
}

// Sorted positions of a block: as many as leave 8 CTAs for each SM.
int block_length(int64_t T, int64_t d) {
  const int64_t chunks = (d + 1023) / 1024, want = T * chunks / (8 * sm_count());
  int n = 4;
  while (n < kBlockMost && n < want) n *= 2;
  return n;
}
int64_t sort_bytes(int64_t T) { return (T * 8 + 255) / 256 * 256; }

int64_t wide_of(int64_t d) {
  const RowThreads r = row_threads(d, kSumThreads);
  return static_cast<int64_t>(r.x) * r.chunks * 8;
}

template <typename Td, typename To, int E>
cudaError_t launch_sums_as(const SumArgs& a, cudaStream_t s) {
  const RowThreads r = row_threads(a.g.d, kSumThreads);
  const int64_t blocks = (a.g.T + a.length - 1) / a.length;
  cudaError_t e = launch_pdl(embed_sum_kernel<Td, To, 4, E>, dim3(static_cast<unsigned>(blocks), r.chunks), dim3(r.x), 0, s, a);
  if (e != cudaSuccess) return e;
  count_launch();
  if (blocks == 1) return e;
  e = launch_pdl(embed_join_kernel<To, E>, dim3(static_cast<unsigned>(std::min<int64_t>(blocks - 1, 65535)), r.chunks),
                 dim3(r.x, kJoinThreads / r.x), 0, s, a);
  if (e == cudaSuccess) count_launch();
  return e;
}
template <typename Td, typename To>
cudaError_t launch_sums(const SumArgs& a, cudaStream_t s) {
  const bool vec = rows_aligned(a.g.dY, a.g.lddy, a.g.dy_dtype) && rows_aligned(a.g.dW, a.g.lddw, a.g.dw_dtype);
  return vec ? launch_sums_as<Td, To, sizeof(Td) == 2 ? piece<Td, To>() : 8>(a, s) : launch_sums_as<Td, To, 1>(a, s);
}

template <typename Tw, typename To>
cudaError_t launch_embed_as(const p24_embed_args& g, cudaStream_t s) {
  const bool vec = rows_aligned(g.W, g.ldw, g.w_dtype) && rows_aligned(g.Y, g.ldy, g.y_dtype);
  const RowThreads r = row_threads(g.d, 256);
  constexpr int E = piece<Tw, To>();
  const dim3 block(r.x, 256 / r.x);
  auto go = [&](auto kern, int u) {
    const int64_t rows = static_cast<int64_t>(u) * block.y;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>((g.T + rows - 1) / rows), r.chunks), block, 0, s, g);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  // 4 rows a thread where that leaves 8 CTAs for each SM
  if (g.T * r.x * r.chunks >= 256 * 8 * 4 * sm_count()) return vec ? go(embed_kernel<Tw, To, 4, E>, 4) : go(embed_kernel<Tw, To, 4, 1>, 4);
  return vec ? go(embed_kernel<Tw, To, 1, E>, 1) : go(embed_kernel<Tw, To, 1, 1>, 1);
}

}  // namespace

size_t embed_bwd_workspace(int64_t T, int64_t d) {
  const int64_t blocks = (T + block_length(T, d) - 1) / block_length(T, d);
  return static_cast<size_t>(2 * sort_bytes(T) + 2 * blocks * wide_of(d) * sizeof(float));
}

cudaError_t launch_embed(const p24_embed_args& g, cudaStream_t s) {
  if (g.w_dtype == P24_BF16) return g.y_dtype == P24_BF16 ? launch_embed_as<bf16, bf16>(g, s) : launch_embed_as<bf16, float>(g, s);
  return g.y_dtype == P24_BF16 ? launch_embed_as<float, bf16>(g, s) : launch_embed_as<float, float>(g, s);
}

cudaError_t launch_embed_bwd(const p24_embed_bwd_args& g, void* ws, cudaStream_t s) {
  if (g.T == 0) return launch_zeros(g, s);
  SumArgs a{g, nullptr, nullptr, wide_of(g.d), block_length(g.T, g.d)};
  int2* first = static_cast<int2*>(ws);
  int2* second = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + sort_bytes(g.T));
  a.sorted = first;
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * sort_bytes(g.T));
  // Few tokens are ranked, up to 4096 where the sort would not be hidden behind the zeros (at 7.5 TB/s): it takes one
  // cluster and leaves the other SMs to them.
  const double zeros_us = g.accumulate ? 0.0 : static_cast<double>(g.V) * g.d * size_of(g.dw_dtype) / 7.5e6;
  cudaError_t e;
  if (g.T <= kRankMost / 2 || (g.T <= kRankMost && zeros_us < 14.0)) {
    const int T = static_cast<int>(g.T), warps = kRankThreads / 32;
    e = launch_pdl(embed_rank_kernel, dim3((T + warps - 1) / warps), dim3(kRankThreads), static_cast<size_t>((T + 127) / 128 * 128) * sizeof(int),
                   s, g.tokens, T, static_cast<int>(g.V), first);
  } else {
    int total = 1;  // of the keys 0..V
    while (g.V >> total) ++total;
    const int passes = (total + kDigit - 1) / kDigit, bits = (total + passes - 1) / passes;
    int slots = 0;
    const size_t smem = sizeof(SortShared);
    e = row_kernel_slots(reinterpret_cast<const void*>(embed_sort_kernel), kSortThreads, kSortCtas, smem, &slots);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kSortCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, embed_sort_kernel, g, bits, passes, first, second);
  }
  if (e != cudaSuccess) return e;
  count_launch();
  if (!g.accumulate && (e = launch_zeros(g, s)) != cudaSuccess) return e;
  if (g.dy_dtype == P24_BF16) return g.dw_dtype == P24_BF16 ? launch_sums<bf16, bf16>(a, s) : launch_sums<bf16, float>(a, s);
  return g.dw_dtype == P24_BF16 ? launch_sums<float, bf16>(a, s) : launch_sums<float, float>(a, s);
}

}  // namespace p24
