// gradnorm_kernels.cu -- the norm over a list of gradient tensors, and the gradients scaled to a largest
// norm.
//
//   norm = sqrt(sum over all tensors and elements of g^2);   g <- g min(1, max_norm / norm)
//
// The bound is memory: 743 MB of bf16 and fp32 in 106 us (7.0 TB/s), scaled into other tensors in 330 in all (6.8). The
// tensors are cut into chunks of 4 to 32 KB; CTA b of a fixed grid takes chunks b, b + grid, ... (a stretch of
// neighbouring ones each read as fast, but scaled 743 MB in 246 us instead of 226). A thread squares and adds the
// elements of a chunk in fp32, and chunks, threads and CTAs are added as pairs of fp32 numbers, a sum and what its
// rounding left (Knuth's two-sum): the number of elements costs no digits. Chunks whose sum lies outside 2^-100 .. 2^88
// (2^38 such sums still fit fp32) are squared and added again in fp64, so neither does their size. (All of it in fp64
// beyond the chunks took 45 us for 72 tensors of 4.8 MB: an SM adds two a clock.) Every sum has a fixed order. The
// scaling pass goes through the chunks from the end, where the first pass left off: what is in L2 still is read from
// there.
#include <algorithm>

#include "stream_rows.cuh"

namespace p24 {
namespace {

constexpr int kThreads = 256, kUnroll = 8, kCtas = 4;  // of an SM
constexpr int64_t kChunk = kThreads * kUnroll;  // 16-byte vectors, at most
constexpr int kMostTable = 850;   // tensors of a launch: its parameters are up to 32 764 bytes
constexpr int kMostCtas = 1024;

// The list goes with the launch: no copy to the device, and a captured graph keeps its own.
struct Entry {
  const uint8_t* p;
  uint8_t* to;
  int64_t n;      // elements
  int32_t chunk;  // the first one
  int32_t f32;
};
template <int N>
struct Table {
  Entry e[N + 1];               // the last has the number of chunks
  uint16_t first[kMostCtas];    // the tensors of chunk b
  uint16_t last[kMostCtas];     // and of chunk chunks - 1 - b
  int32_t vecs;                 // 16-byte vectors of a chunk
  int32_t count, chunks, ctas;
};

static_assert(sizeof(Table<kMostTable>) + 64 <= 32764, "a launch's parameters");

struct Piece {  // a chunk of a tensor
  const uint8_t* p;
  uint8_t* to;
  int64_t n, vec0;        // elements of the tensor; the chunk's first vector
  int vecs;               // and how many it has
  int head, tail, f32;    // elements before the tensor's first 16-byte boundary and after its last one
  bool first;             // takes those
};

// Chunk c, which is tensor at's, or kUp one's behind it, else before it. (A search from the list's beginning went
// through the launch's constants one miss at a time, 13 us for 72 tensors of 600 KB in all.)
template <bool kUp, int N>
__device__ __forceinline__ Piece piece_of(const Table<N>& t, int c, int& at) {
  if (kUp ? c >= t.e[at + 1].chunk : c < t.e[at].chunk) {
    int step = 1;
    if (kUp) {
      for (; at + step < t.count && c >= t.e[at + step].chunk; step *= 2) at += step;
    } else {
      for (; at - step > 0 && c < t.e[at - step + 1].chunk; step *= 2) at -= step;
    }
    int lo = kUp ? at : max(at - step, 0), hi = kUp ? min(at + step, t.count) : at + 1;  // the tensor is in [lo, hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.e[mid].chunk <= c) lo = mid;
      else hi = mid;
    }
    at = lo;
  }
  const Entry& e = t.e[at];
  Piece r;
  r.p = e.p, r.to = e.to, r.n = e.n, r.f32 = e.f32;
  const int shift = r.f32 ? 2 : 1;
  r.head = static_cast<int>(min(r.n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(r.p) & 15u)) & 15u) >> shift)));
  const int64_t all = (r.n - r.head) << shift >> 4;
  r.tail = static_cast<int>(r.n - r.head - (all << 4 >> shift));
  r.vec0 = static_cast<int64_t>(c - e.chunk) * t.vecs;
  r.vecs = static_cast<int>(min(all - r.vec0, static_cast<int64_t>(t.vecs)));
  r.first = r.vec0 == 0;
  return r;
}
__device__ __forceinline__ float element(const Piece& r, int64_t i) {
  return r.f32 ? reinterpret_cast<const float*>(r.p)[i] : to_float(reinterpret_cast<const bf16*>(r.p)[i]);
}

__device__ __forceinline__ void words8(const uint4& q, bool f32, float (&v)[8]) {
  if (f32) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    v[4] = v[5] = v[6] = v[7] = 0.f;
  } else {
    widen(q.x, v[0], v[1]);
    widen(q.y, v[2], v[3]);
    widen(q.z, v[4], v[5]);
    widen(q.w, v[6], v[7]);
  }
}

// A sum and what its rounding left.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(const Pair& a, const Pair& b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

// What a CTA, or all of them, come to: the sum of the chunks in range, and of the others.
struct Sum {
  Pair in;
  double out;
};
struct SumShared {
  Pair in[kThreads / 32];
  double out[kThreads / 32];
};
// Over the CTA, in every thread.
__device__ __forceinline__ Sum cta_sum(Sum x, SumShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a bit pattern other than 0: a number, or NaN
  const bool rare = __syncthreads_or(__double_as_longlong(x.out) != 0);
#pragma unroll
  for (int i = 16; i; i >>= 1) x.in = add(x.in, Pair{__shfl_xor_sync(~0u, x.in.hi, i), __shfl_xor_sync(~0u, x.in.lo, i)});
  if (lane == 0) sh.in[warp] = x.in;
  if (rare) {
#pragma unroll 1
    for (int i = 16; i; i >>= 1) x.out += __shfl_xor_sync(~0u, x.out, i);
    if (lane == 0) sh.out[warp] = x.out;
  }
  __syncthreads();
  Sum y{sh.in[0], 0.0};
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) y.in = add(y.in, sh.in[i]);
  if (rare)
#pragma unroll 1
    for (int i = 0; i < kThreads / 32; ++i) y.out += sh.out[i];
  return y;
}
__device__ __forceinline__ float root(const Sum& s) {
  if (__double_as_longlong(s.out) == 0) return sqrtf(__fadd_rn(s.in.hi, s.in.lo));
  return static_cast<float>(sqrt(s.out + s.in.hi + s.in.lo));
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas) grad_squares_kernel(const __grid_constant__ Table<N> t, Sum* sums) {
  __shared__ SumShared sh;
  int at = t.first[blockIdx.x];
  pdl_wait();
  pdl_trigger();
  Sum total{Pair{0.f, 0.f}, 0.0};
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Piece r = piece_of<true>(t, c, at);
    const uint4* q = reinterpret_cast<const uint4*>(r.p + (r.head << (r.f32 ? 2 : 1))) + r.vec0;
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * kThreads + threadIdx.x;
      x[u] = i < r.vecs ? q[i] : make_uint4(0, 0, 0, 0);
    }
    float edge = 0.f;
    if (r.first && threadIdx.x < r.head + r.tail)
      edge = element(r, threadIdx.x < r.head ? threadIdx.x : r.n - r.tail + threadIdx.x - r.head);
    float s0 = edge * edge, s1 = 0.f;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[8];
      words8(x[u], r.f32, v);
#pragma unroll
      for (int k = 0; k < 8; k += 2) s0 = fmaf(v[k], v[k], s0), s1 = fmaf(v[k + 1], v[k + 1], s1);
    }
    const float s = s0 + s1;
    if (s >= 0x1p-100f && s <= 0x1p88f) {
      total.in = add(total.in, Pair{s, 0.f});
      continue;
    }
    // only zeros, or squares that fp32 does not hold, or no numbers
    uint32_t any = __float_as_uint(edge);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) any |= x[u].x | x[u].y | x[u].z | x[u].w;
    if ((any & (r.f32 ? 0x7fffffffu : 0x7fff7fffu)) == 0) continue;
    total.out += static_cast<double>(edge) * edge;
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * kThreads + threadIdx.x;
      float v[8];
      words8(i < r.vecs ? q[i] : make_uint4(0, 0, 0, 0), r.f32, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) total.out += static_cast<double>(v[k]) * v[k];
    }
  }
  total = cta_sum(total, sh);
  if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

// The norm of `n` CTAs' sums, in every thread.
__device__ __forceinline__ float norm_of(const Sum* sums, int n, SumShared& sh) {
  Sum x{Pair{0.f, 0.f}, 0.0};
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Sum y = sums[i];
    x.in = add(x.in, y.in);
    if (__double_as_longlong(y.out) != 0) x.out += y.out;
  }
  return root(cta_sum(x, sh));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const Sum* sums, int n, float* norm) {
  __shared__ SumShared sh;
  pdl_wait();
  pdl_trigger();
  const float x = norm_of(sums, n, sh);
  if (threadIdx.x == 0) *norm = x;
}

// kLong: a CTA a chunk, started by the hardware in the order of memory, and the norm is there already. Else the CTAs that
// run at once take the chunks in turn, and each finds the norm from the sums: a launch less. (743 MB 348 us by CTAs that
// stay, 342 by 4 times as many, 330 by one a chunk; 84 MB 36 either way, 16 MB 10.9 and 11.3.)
constexpr int64_t kLongBytes = 80 << 20;
template <int N, bool kLong>
__global__ void __launch_bounds__(kThreads, kCtas) grad_scale_kernel(const __grid_constant__ Table<N> t, const Sum* sums, int n,
                                                              float max_norm, float* norm) {
  __shared__ SumShared sh;
  int at = 0;
  if (kLong) {
    for (int hi = t.count; hi - at > 1;) {
      const int mid = (at + hi) >> 1;
      if (t.e[mid].chunk <= t.chunks - 1 - static_cast<int>(blockIdx.x)) at = mid;
      else hi = mid;
    }
  } else {
    at = t.last[blockIdx.x];
  }
  pdl_wait();
  pdl_trigger();
  const float x = kLong ? *norm : norm_of(sums, n, sh);
  if (!kLong && norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = x;
  const bool over = x > max_norm && x < __int_as_float(0x7f800000);  // a norm that is no number scales nothing
  const float f = over ? max_norm / x : 1.f;
  for (int c = t.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Piece r = piece_of<false>(t, c, at);
    if (!over && r.to == r.p) continue;
    const int shift = r.f32 ? 2 : 1;
    const uint4* q = reinterpret_cast<const uint4*>(r.p + (r.head << shift)) + r.vec0;
    uint8_t* to = r.to + (r.head << shift) + (r.vec0 << 4);
    const bool vec = (reinterpret_cast<uintptr_t>(to) & 15u) == 0;
    uint4 y[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * kThreads + threadIdx.x;
      if (i < r.vecs) y[u] = q[i];
    }
    if (r.first && threadIdx.x < r.head + r.tail) {
      const int64_t i = threadIdx.x < r.head ? threadIdx.x : r.n - r.tail + threadIdx.x - r.head;
      const float e = element(r, i) * f;
      if (r.f32) reinterpret_cast<float*>(r.to)[i] = e;
      else reinterpret_cast<bf16*>(r.to)[i] = static_cast<bf16>(e);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = u * kThreads + threadIdx.x;
      if (i >= r.vecs) continue;
      float v[8];
      words8(y[u], r.f32, v);
      uint4 o;
      if (r.f32)
        o = make_uint4(__float_as_uint(v[0] * f), __float_as_uint(v[1] * f), __float_as_uint(v[2] * f), __float_as_uint(v[3] * f));
      else
        o = make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f), pack_bf16x2(v[4] * f, v[5] * f),
                       pack_bf16x2(v[6] * f, v[7] * f));
      if (vec) {
        reinterpret_cast<uint4*>(to)[i] = o;
      } else if (r.f32) {
        uint32_t* w = reinterpret_cast<uint32_t*>(to) + 4 * i;
        w[0] = o.x, w[1] = o.y, w[2] = o.z, w[3] = o.w;
      } else {
        uint16_t* w = reinterpret_cast<uint16_t*>(to) + 8 * i;
        const uint32_t h[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = static_cast<uint16_t>(h[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
}

// As many as run at once.
int64_t grid_most() { return std::min<int64_t>(kMostCtas, sm_count() * kCtas); }

int64_t chunks_of(const p24_tensor& t, int64_t most) {
  const int64_t size = t.dtype == P24_F32 ? 4 : 2;
  const int64_t head = std::min<int64_t>(t.n, ((16 - (reinterpret_cast<uintptr_t>(t.p) & 15u)) & 15u) / size);
  const int64_t vecs = (t.n - head) * size / 16;
  return t.n == 0 ? 0 : std::max<int64_t>(1, (vecs + most - 1) / most);
}

// Tensors [from, ...) of the list, as many as one launch takes; returns where the next one goes on.
template <int N>
int64_t fill_table(Table<N>& t, const p24_tensor* g, const p24_tensor* out, int64_t n, int64_t from) {
  int64_t chunks = 0, bytes = 0, i = from;
  int count = 0;
  for (int64_t k = from; k < std::min<int64_t>(n, from + N); ++k) bytes += g[k].n * (g[k].dtype == P24_F32 ? 4 : 2);
  // chunks as long as leaves each CTA some
  int64_t vecs = kChunk;
  while (vecs > kThreads && bytes < vecs * 16 * grid_most()) vecs /= 2;
  t.vecs = static_cast<int32_t>(vecs);
  for (; i < n && count < N; ++i) {
    const int64_t c = chunks_of(g[i], vecs);
    if (c == 0) continue;
    t.e[count++] = Entry{static_cast<const uint8_t*>(g[i].p), static_cast<uint8_t*>(out ? out[i].p : g[i].p), g[i].n,
                         static_cast<int32_t>(chunks), g[i].dtype == P24_F32};
    chunks += c;
  }
  t.e[count].chunk = t.chunks = static_cast<int32_t>(chunks);
  t.ctas = static_cast<int32_t>(std::min<int64_t>(chunks, grid_most()));
  t.count = count;
  for (int b = 0, up = 0, down = count - 1; b < t.ctas; ++b) {
    while (b >= t.e[up + 1].chunk) ++up;
    while (chunks - 1 - b < t.e[down].chunk) --down;
    t.first[b] = static_cast<uint16_t>(up);
    t.last[b] = static_cast<uint16_t>(down);
  }
  return i;
}

template <int N>
cudaError_t run_list(const p24_tensor* g, const p24_tensor* out, int64_t n, bool scale, float max_norm, float* norm, Sum* sums,
                     cudaStream_t s) {
  Table<N> t;
  int64_t used = 0, bytes = 0;
  cudaError_t e;
  for (int64_t i = 0; i < n;) {
    i = fill_table(t, g, nullptr, n, i);
    if (t.chunks == 0) continue;
    e = launch_pdl(grad_squares_kernel<N>, dim3(static_cast<unsigned>(t.ctas)), dim3(kThreads), 0, s, t, sums + used);
    if (e != cudaSuccess) return e;
    count_launch();
    used += t.ctas;
    bytes += static_cast<int64_t>(t.chunks) * t.vecs * 16;
  }
  const bool longer = scale && bytes > kLongBytes;
  if (longer && !norm) norm = reinterpret_cast<float*>(sums + used);
  if ((!scale || longer || used == 0) && norm) {
    e = launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const Sum*>(sums), static_cast<int>(used), norm);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  for (int64_t i = scale && used > 0 ? 0 : n; i < n;) {
    i = fill_table(t, g, out, n, i);
    if (t.chunks == 0) continue;
    const auto kern = longer ? grad_scale_kernel<N, true> : grad_scale_kernel<N, false>;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(longer ? t.chunks : t.ctas)), dim3(kThreads), 0, s, t, static_cast<const Sum*>(sums),
                   static_cast<int>(used), max_norm, norm);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaSuccess;
}

}  // namespace

// A sum for each CTA of the launches that a list of n tensors takes, and one for the norm where there is no place for it.
size_t grad_norm_workspace(int64_t n) {
  return static_cast<size_t>(std::max<int64_t>(1, (n + kMostTable - 1) / kMostTable) * grid_most() + 1) * sizeof(Sum);
}

cudaError_t launch_grad_norm(const p24_tensor* g, const p24_tensor* out, int64_t n, bool scale, float max_norm, float* norm,
                             void* ws, cudaStream_t s) {
  Sum* sums = static_cast<Sum*>(ws);
  if (n <= 16) return run_list<16>(g, out, n, scale, max_norm, norm, sums, s);
  if (n <= 128) return run_list<128>(g, out, n, scale, max_norm, norm, sums, s);
  return run_list<kMostTable>(g, out, n, scale, max_norm, norm, sums, s);
}

}  // namespace p24
