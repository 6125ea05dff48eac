// gradnorm_kernels.cu -- the norm over a list of gradient tensors, and the gradients scaled to a largest
// norm.
//
//   norm = sqrt(sum over all tensors and elements of g^2);   g <- g min(1, max_norm / norm)
//
// The tensors are cut into chunks of 32 KB; CTA b of a fixed grid takes chunks b, b + grid, ... A thread
// squares and adds the elements of a chunk in fp32 and the chunks' sums in fp64, so neither the number
// of elements nor their size (squares outside fp32 are summed again in fp64) costs digits, and every sum
// has a fixed order. The scaling pass goes through the chunks from the end, where the first pass left
// off: what still is in L2 is read from there.
#include <algorithm>

#include "stream_rows.cuh"

namespace p24 {
namespace {

constexpr int kThreads = 256, kUnroll = 8;
constexpr int64_t kChunk = kThreads * kUnroll;  // 16-byte vectors

// The list goes with the launch: no copy to the device, and a captured graph keeps its own.
template <int N>
struct Table {
  const void* p[N];
  void* to[N];
  int64_t n[N];
  int32_t chunk[N + 1];  // the first chunk of each tensor; past the last: all chunks
  uint8_t dtype[N];
  int32_t count;
};

struct Piece {  // a chunk of a tensor
  const uint8_t* p;
  uint8_t* to;
  int64_t n, vec0, vecs;  // elements; the chunk's first vector and how many it has
  int head, tail, f32;    // elements before the tensor's first 16-byte boundary and after its last one
  bool first;             // takes those
};

template <int N>
__device__ __forceinline__ Piece piece_of(const Table<N>& t, int chunk, int& at) {
  while (chunk < t.chunk[at]) --at;
  while (chunk >= t.chunk[at + 1]) ++at;
  Piece r;
  r.p = static_cast<const uint8_t*>(t.p[at]);
  r.to = static_cast<uint8_t*>(t.to[at]);
  r.n = t.n[at];
  r.f32 = t.dtype[at] == P24_F32;
  const int shift = r.f32 ? 2 : 1;
  r.head = static_cast<int>(min(r.n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(r.p) & 15u)) & 15u) >> shift)));
  const int64_t all = (r.n - r.head) << shift >> 4;
  r.tail = static_cast<int>(r.n - r.head - (all << 4 >> shift));
  r.vec0 = (chunk - t.chunk[at]) * kChunk;
  r.vecs = min(all - r.vec0, kChunk);
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

// The sum over a CTA in thread 0, in a fixed order.
__device__ __forceinline__ double cta_sum(double x, double* sh) {
#pragma unroll
  for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) x += sh[i];
  return x;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Table<N> t, double* sums) {
  __shared__ double sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  double total = 0;
  int at = 0;
  for (int c = blockIdx.x; c < t.chunk[t.count]; c += gridDim.x) {
    const Piece r = piece_of(t, c, at);
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
    if (s >= 0x1p-100f && s < __int_as_float(0x7f800000)) {
      total += s;
    } else {  // zeros, or squares that fp32 does not hold
      total += static_cast<double>(edge) * edge;
#pragma unroll 1
      for (int u = 0; u < kUnroll; ++u) {
        const int i = u * kThreads + threadIdx.x;
        float v[8];
        words8(i < r.vecs ? q[i] : make_uint4(0, 0, 0, 0), r.f32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (v[k] != 0.f) total += static_cast<double>(v[k]) * v[k];
      }
    }
  }
  total = cta_sum(total, sh);
  if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

// The norm of `n` CTAs' sums, in every thread.
__device__ __forceinline__ float norm_of(const double* sums, int n, double* sh) {
  double x = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) x += sums[i];
  return static_cast<float>(sqrt(cta_sum(x, sh)));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* sums, int n, float* norm) {
  __shared__ double sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const float x = norm_of(sums, n, sh);
  if (threadIdx.x == 0) *norm = x;
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Table<N> t, const double* sums, int n,
                                                              float max_norm, float* norm) {
  __shared__ double sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const float x = norm_of(sums, n, sh);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = x;
  const bool over = x > max_norm && x < __int_as_float(0x7f800000);  // a norm that is no number scales nothing
  const float f = over ? max_norm / x : 1.f;
  int at = t.count - 1;
  for (int c = t.chunk[t.count] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Piece r = piece_of(t, c, at);
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

constexpr int kMostTable = 900;
int64_t grid_most() { return sm_count() * 6; }

int64_t chunks_of(const p24_tensor& t) {
  const int64_t size = t.dtype == P24_F32 ? 4 : 2;
  const int64_t head = std::min<int64_t>(t.n, ((16 - (reinterpret_cast<uintptr_t>(t.p) & 15u)) & 15u) / size);
  const int64_t vecs = (t.n - head) * size / 16;
  return t.n == 0 ? 0 : std::max<int64_t>(1, (vecs + kChunk - 1) / kChunk);
}

// Tensors [from, ...) of the list, as many as one launch takes.
template <int N>
int64_t fill_table(Table<N>& t, const p24_tensor* g, const p24_tensor* out, int64_t n, int64_t from) {
  int64_t chunks = 0, i = from;
  t.count = 0;
  for (; i < n && t.count < N; ++i) {
    const int64_t c = chunks_of(g[i]);
    if (c == 0) continue;
    t.p[t.count] = g[i].p;
    t.to[t.count] = out ? out[i].p : const_cast<void*>(static_cast<const void*>(g[i].p));
    t.n[t.count] = g[i].n;
    t.dtype[t.count] = static_cast<uint8_t>(g[i].dtype);
    t.chunk[t.count++] = static_cast<int32_t>(chunks);
    chunks += c;
  }
  t.chunk[t.count] = static_cast<int32_t>(chunks);
  return i;
}

template <int N>
cudaError_t run_list(const p24_tensor* g, const p24_tensor* out, int64_t n, bool scale, float max_norm, float* norm, double* sums,
                     cudaStream_t s) {
  Table<N> t;
  int64_t used = 0;
  cudaError_t e;
  for (int64_t i = 0; i < n;) {
    i = fill_table(t, g, nullptr, n, i);
    if (t.count == 0) continue;
    const int64_t grid = std::min<int64_t>(t.chunk[t.count], grid_most());
    e = launch_pdl(grad_squares_kernel<N>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, t, sums + used);
    if (e != cudaSuccess) return e;
    count_launch();
    used += grid;
  }
  if (scale && used > 0) {
    for (int64_t i = 0; i < n;) {
      i = fill_table(t, g, out, n, i);
      if (t.count == 0) continue;
      const int64_t grid = std::min<int64_t>(t.chunk[t.count], grid_most());
      e = launch_pdl(grad_scale_kernel<N>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, t, static_cast<const double*>(sums),
                     static_cast<int>(used), max_norm, norm);
      if (e != cudaSuccess) return e;
      count_launch();
    }
    return cudaSuccess;
  }
  if (!norm) return cudaSuccess;  // an empty list, and no norm asked for
  e = launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(sums), static_cast<int>(used), norm);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

// A sum for each CTA of the launches that a list of n tensors takes.
size_t grad_norm_workspace(int64_t n) {
  return static_cast<size_t>(std::max<int64_t>(1, (n + kMostTable - 1) / kMostTable) * grid_most()) * sizeof(double);
}

cudaError_t launch_grad_norm(const p24_tensor* g, const p24_tensor* out, int64_t n, bool scale, float max_norm, float* norm,
                             void* ws, cudaStream_t s) {
  double* sums = static_cast<double*>(ws);
  if (n <= 16) return run_list<16>(g, out, n, scale, max_norm, norm, sums, s);
  if (n <= 128) return run_list<128>(g, out, n, scale, max_norm, norm, sums, s);
  return run_list<kMostTable>(g, out, n, scale, max_norm, norm, sums, s);
}

}  // namespace p24
