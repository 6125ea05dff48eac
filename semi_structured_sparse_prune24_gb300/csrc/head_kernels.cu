// head_kernels.cu -- the language-model head's row operators: token log probabilities
// (with entropy and the top alternatives), distillation from a teacher's top-K list, and
// the gradients of both. All of them walk rows of logits z [T, V] (bf16 or fp32), one CTA
// per row; sums, maxima and statistics are fp32.
//
//   x = (z - m) / tau,  m = max z,  s = sum exp(x),  p = exp(x) / s
//   logp = x[token] - ln s        H = ln s - (1/s) sum exp(x) x
//
// Rows are read as 16-byte vectors aligned in memory, whatever the row's own alignment:
// vector v of a row covers elements [v * N - a, (v + 1) * N - a), a = elements between the
// preceding 16-byte boundary and the row's start; the first and last vector may be partial
// and are then read element by element, never outside the row.
//
// Bound: HBM, one read of the row (forward), one read and one write (gradients).
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "p24_internal.h"
#include "p24_ptx.cuh"

namespace p24 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTopMax = P24_TOPK_MAX;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(x, floor) that keeps a NaN. The floor of -1e30 makes exp(x) of -inf (a masked logit) 0
// and the product exp(x) * x as well, where -inf would give 0 * inf.
__device__ __forceinline__ float floored(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fF149F2CA;" : "=f"(y) : "f"(x));  // -1e30
  return y;
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};

// Elements [i0, i0 + N) of a row of V; the ones outside it read as -inf. i0 is a vector's
// first element: the 16-byte load is aligned.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int i0, int V, float (&x)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  if (i0 >= 0 && i0 <= V - N) {
    const uint4 r = *reinterpret_cast<const uint4*>(row + i0);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j;
      x[j] = (i >= 0 && i < V) ? to_f32(row[i]) : ninf();
    }
  }
}

// Elements [i0, i0 + N) of an output row; `vec`: the output row has the input row's alignment.
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int i0, int V, bool vec, const float (&x)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  if (vec && i0 >= 0 && i0 <= V - N) {
    uint4 r;
    if constexpr (sizeof(T) == 2) {
      r = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    } else {
      r = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    *reinterpret_cast<uint4*>(row + i0) = r;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j;
      if (i >= 0 && i < V) row[i] = static_cast<T>(x[j]);
    }
  }
}

template <typename T>
__device__ __forceinline__ int misaligned(const T* row) {  // elements past the preceding 16-byte boundary
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// ---------------------------------------------------------------- row sums
// The running sums of a softmax over part of a row, relative to the part's maximum m:
// s = sum exp((z - m)/tau), a = sum exp((z - m)/tau) (z - m). s == 0: nothing above -inf yet.
struct Sums {
  float m, s, a;
};

// Move the sums to the reference `to` >= m. c = log2(e) / tau.
__device__ __forceinline__ void rebase(Sums& u, float to, float c) {
  if (u.s != 0.f) {
    const float d = floored(u.m - to);
    const float r = ex2(d * c);
    u.a = (u.a + u.s * d) * r;
    u.s *= r;
  }
  u.m = to;
}

__device__ __forceinline__ Sums join(Sums u, Sums v, float c) {
  const float m = fmaxf(u.m, v.m);
  rebase(u, m, c);
  rebase(v, m, c);
  return Sums{m, u.s + v.s, u.a + v.a};
}

template <bool kEntropy, int N>
__device__ __forceinline__ void add_vec(Sums& u, const float (&x)[N], float c) {
  float vm = x[0];
#pragma unroll
  for (int j = 1; j < N; ++j) vm = fmaxf(vm, x[j]);
  if (vm > u.m) rebase(u, vm, c);
  const float ref = u.m == ninf() ? 0.f : u.m;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float t = floored(x[j] - ref);
    const float e = ex2(t * c);
    u.s += e;
    if constexpr (kEntropy) u.a = fmaf(e, t, u.a);
  }
}

// The CTA's sums, in every thread. buf: kWarps entries. Fixed order: repeated calls agree bit for bit.
__device__ __forceinline__ Sums block_join(Sums u, float c, Sums* buf) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Sums v{__shfl_xor_sync(~0u, u.m, d), __shfl_xor_sync(~0u, u.s, d), __shfl_xor_sync(~0u, u.a, d)};
    u = join(u, v, c);
  }
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = u;
  __syncthreads();
  u = buf[0];
  for (int w = 1; w < kWarps; ++w) u = join(u, buf[w], c);
  return u;
}

// ---------------------------------------------------------------- top k
// Order of the logits as an unsigned key: larger key first; NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Key and position in one number that orders both: ties go to the lower position.
__device__ __forceinline__ uint64_t entry(uint32_t key, int i) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int entry_pos(uint64_t e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }

struct TopShared {
  uint32_t hist[256];
  int warp[kWarps];
  uint32_t prefix;
  int left;   // how many of the elements equal to the prefix are still to be taken
  int n;      // entries collected
  uint64_t list[kTopMax];
};

// The k first elements of the row (k <= V), unordered, into sh.list: a radix selection
// of the k-th key, 8 bits a pass, then the elements above it and, in order of position,
// as many equal to it as are needed.
template <typename T>
__device__ void select_exact(const T* row, int a, int nvec, int V, int k, TopShared& sh) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh.prefix = 0;
    sh.left = k;
    sh.n = 0;
  }
  uint32_t mask = 0;
  for (int shift = 24; shift >= 32 - 8 * static_cast<int>(sizeof(T)); shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = sh.prefix;
    for (int v = tid; v < nvec; v += kThreads) {
      float x[N];
      load_vec(row, v * N - a, V, x);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = v * N - a + j;
        const uint32_t key = order_key(x[j]);
        if (i >= 0 && i < V && (key & mask) == prefix) atomicAdd(&sh.hist[(key >> shift) & 255u], 1u);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int left = sh.left, d = 255;
      while (d > 0 && static_cast<int>(sh.hist[d]) < left) left -= static_cast<int>(sh.hist[d--]);
      sh.left = left;
      sh.prefix = prefix | (static_cast<uint32_t>(d) << shift);
    }
    mask |= 255u << shift;
    __syncthreads();
  }
  const uint32_t kth = sh.prefix;
  const int left = sh.left;
  int equal_before = 0;
  for (int v0 = 0; v0 < nvec; v0 += kThreads) {
    const int v = v0 + tid;
    float x[N];
    uint32_t eq = 0;
    if (v < nvec) {
      load_vec(row, v * N - a, V, x);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = v * N - a + j;
        if (i < 0 || i >= V) continue;
        const uint32_t key = order_key(x[j]);
        if ((key & mask) > kth) sh.list[atomicAdd(&sh.n, 1)] = entry(key, i);
        if ((key & mask) == kth) eq |= 1u << j;
      }
    }
    // position of this thread's equal elements among all of the row's
    int mine = __popc(eq), incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, incl, d);
      if ((tid & 31) >= d) incl += y;
    }
    if ((tid & 31) == 31) sh.warp[tid >> 5] = incl;
    __syncthreads();
    int before = equal_before + incl - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < (tid >> 5)) before += sh.warp[w];
      total += sh.warp[w];
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if ((eq >> j) & 1u) {
        if (before < left) sh.list[k - left + before] = entry(order_key(x[j]), v * N - a + j);
        ++before;
      }
    equal_before += total;
    __syncthreads();
  }
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const p24_logprobs_args g) {
  constexpr int N = Vec<T>::N;
  __shared__ Sums sums[kWarps];
  __shared__ TopShared sh;
  const int tid = threadIdx.x, V = static_cast<int>(g.V);
  const int64_t t = blockIdx.x;
  const T* row = static_cast<const T*>(g.logits) + t * g.ldz;
  const int a = misaligned(row);
  const int nvec = static_cast<int>((static_cast<int64_t>(V) + a + N - 1) / N);
  const float c = kLog2e / g.temperature;
  Sums u{ninf(), 0.f, 0.f};
  for (int v = tid; v < nvec; v += kThreads) {
    float x[N];
    load_vec(row, v * N - a, V, x);
    add_vec<kEntropy>(u, x, c);
  }
  u = block_join(u, c, sums);
  const float ls = u.s == 0.f ? ninf() : logf(u.s);
  // ln of the probability of a logit; a row with nothing above -inf has none
  auto logp = [&](float z) { return u.s == 0.f ? ninf() : (z - u.m) / g.temperature - ls; };
  if (tid == 0) {
    if (g.stats) {
      g.stats[2 * t] = u.m;
      g.stats[2 * t + 1] = ls;
    }
    if (g.logp) {
      const int tok = g.tokens[t];
      g.logp[t] = (tok >= 0 && tok < V) ? logp(to_f32(row[tok])) : 0.f;
    }
    if (kEntropy) g.entropy[t] = u.s == 0.f ? 0.f : ls - u.a / (u.s * g.temperature);
  }
  if (g.k == 0) return;
  const int K = static_cast<int>(g.k), k = K < V ? K : V;
  __syncthreads();
  select_exact(row, a, nvec, V, k, sh);
  float* top_logp = g.top_logp + t * K;
  int32_t* top_idx = g.top_idx + t * K;
  if (tid < K) {
    if (tid < k) {
      const uint64_t e = sh.list[tid];
      int rank = 0;
      for (int j = 0; j < k; ++j) rank += sh.list[j] > e;
      const int i = entry_pos(e);
      top_idx[rank] = i;
      top_logp[rank] = logp(to_f32(row[i]));
    } else {
      top_idx[tid] = -1;
      top_logp[tid] = ninf();
    }
  }
}

// dz = (1/tau) [ dlogp (delta - p) - dentropy p (ln p + H) ]
template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kThreads) logprobs_bwd_kernel(const p24_logprobs_args g) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, V = static_cast<int>(g.V);
  const int64_t t = blockIdx.x;
  const T* row = static_cast<const T*>(g.logits) + t * g.ldz;
  T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
  const int a = misaligned(row);
  const bool vec = misaligned(out) == a;
  const int nvec = static_cast<int>((static_cast<int64_t>(V) + a + N - 1) / N);
  const int tok = g.tokens ? g.tokens[t] : -1;
  const float m = g.stats[2 * t], ls = g.stats[2 * t + 1];
  const float dl = (g.dlogp && tok >= 0 && tok < V) ? g.dlogp[t] / g.temperature : 0.f;
  const float dh = kEntropy ? g.dentropy[t] / g.temperature : 0.f;
  const float c = 1.f / g.temperature;
  const float k0 = kEntropy ? -(dl + dh * g.entropy[t]) : -dl;  // dz = p (k0 - dh ln p) + dl delta
  const bool none = m == ninf();
  for (int v = tid; v < nvec; v += kThreads) {
    const int i0 = v * N - a;
    float x[N], d[N];
    load_vec(row, i0, V, x);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float lp = floored((x[j] - m) * c - ls);
      d[j] = none ? 0.f : ex2(lp * kLog2e) * (kEntropy ? fmaf(-dh, lp, k0) : k0);
      if (i0 + j == tok && !none) d[j] += dl;
    }
    store_vec(out, i0, V, vec, d);
  }
}

// ---------------------------------------------------------------- distillation
struct DistillShared {
  Sums sums[kWarps], sums1[kWarps];
  int idx[kTopMax];      // listed column, or -1
  float z[kTopMax];      // the student's logit there
  float q[kTopMax];      // the teacher's probability
  float q_sum, q_rest;
  float kl;
  int label_listed;
};

// kMode 0: loss and statistics; 1: loss, statistics and gradient; 2: gradient from saved statistics.
// kTwo: the label's softmax (temperature 1) differs from the list's.
template <typename T, bool kTwo, int kMode>
__global__ void __launch_bounds__(kThreads) distill_kernel(const p24_distill_args g) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint32_t listed[];  // tail: a byte per vector, bit j set where element j is listed
  __shared__ DistillShared sh;
  const int tid = threadIdx.x, V = static_cast<int>(g.V), K = static_cast<int>(g.K);
  const int64_t t = blockIdx.x;
  const T* row = static_cast<const T*>(g.logits) + t * g.ldz;
  const int a = misaligned(row);
  const int nvec = static_cast<int>((static_cast<int64_t>(V) + a + N - 1) / N);
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  const float tau = g.temperature, c = kLog2e / tau;
  const int label = g.labels ? g.labels[t] : -1;
  const bool has_label = label >= 0 && label < V;
  const float z_label = has_label ? to_f32(row[label]) : 0.f;  // read before an in-place gradient overwrites it

  // the teacher's list
  if (tid == 0) sh.label_listed = 0;
  if (tid < K) {
    const int i = g.top_idx[t * K + tid];
    const bool on = i >= 0 && i < V;
    sh.idx[tid] = on ? i : -1;
    sh.z[tid] = on ? to_f32(row[i]) : ninf();
    sh.q[tid] = on ? g.top_val[t * K + tid] : ninf();
  }
  if (kMode != 2 && tail)
    for (int w = tid; w < (nvec + 3) / 4; w += kThreads) listed[w] = 0;
  __syncthreads();
  if (kMode != 2 && tail && tid < K && sh.idx[tid] >= 0) {
    const int e = sh.idx[tid] + a, v = e / N;
    atomicOr(&listed[v >> 2], 1u << (8 * (v & 3) + e % N));
  }
  if (tid < K && sh.idx[tid] == label) sh.label_listed = 1;
  if (tid < 32) {
    // q: softmax of the listed values at the temperature, or (tail) the probabilities they stand for
    float top = ninf(), sum = 0.f;
    for (int j = tid; j < K; j += 32) top = fmaxf(top, sh.q[j]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const bool some = top > ninf();
    for (int j = tid; j < K; j += 32) {
      const float x = sh.q[j];
      const float q = sh.idx[j] < 0 ? 0.f : x != x ? x : tail ? expf(x) : some ? expf((x - top) / tau) : 0.f;
      sh.q[j] = q;
      sum += q;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if (!tail)
      for (int j = tid; j < K; j += 32) sh.q[j] = sum != 0.f ? sh.q[j] / sum : 0.f;
    if (tid == 0) {
      sh.q_rest = tail ? fmaxf(1.f - sum, 0.f) : 0.f;
      sh.q_sum = tail ? sum : sum != 0.f ? 1.f : 0.f;
    }
  }
  __syncthreads();

  float m, ls, lr, l1;  // maximum, ln of the sums: all, not listed, all at temperature 1
  if constexpr (kMode == 2) {
    m = g.stats[4 * t], ls = g.stats[4 * t + 1], lr = g.stats[4 * t + 2], l1 = g.stats[4 * t + 3];
  } else {
    Sums u{ninf(), 0.f, 0.f}, u1{ninf(), 0.f, 0.f};
    float top = ninf();  // sums of the listed elements are added at the end (tail)
    for (int v = tid; v < nvec; v += kThreads) {
      float x[N];
      load_vec(row, v * N - a, V, x);
      if (kTwo) add_vec<false>(u1, x, kLog2e);
      if (tail) {
        const uint32_t b = (listed[v >> 2] >> (8 * (v & 3))) & 255u;
        if (b) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if ((b >> j) & 1u) x[j] = ninf();
        }
      }
      add_vec<false>(u, x, c);
    }
    u = block_join(u, c, sh.sums);
    if (kTwo) u1 = block_join(u1, kLog2e, sh.sums1);
    Sums rest = u;
    if (tail) {
      for (int j = 0; j < K; ++j) top = fmaxf(top, sh.z[j]);
      const float to = fmaxf(u.m, top);
      rebase(u, to, c);
      rest = u;
      if (to > ninf())
        for (int j = 0; j < K; ++j) u.s += ex2(floored(sh.z[j] - to) * c);
    }
    m = u.m;
    ls = u.s == 0.f ? ninf() : logf(u.s);
    lr = !tail ? 0.f : rest.s == 0.f ? ninf() : logf(rest.s);
    l1 = !g.labels ? 0.f : !kTwo ? ls : u1.s == 0.f ? ninf() : logf(u1.s);
    if (tid < 32) {
      float kl = 0.f;
      for (int j = tid; j < K; j += 32) {
        const float q = sh.q[j];
        const float lp = u.s == 0.f ? ninf() : (sh.z[j] - m) / tau - ls;
        if (q != 0.f) kl += q * (logf(q) - lp);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) kl += __shfl_xor_sync(~0u, kl, d);
      if (tid == 0) {
        const float qr = lr == ninf() ? 0.f : sh.q_rest;
        if (qr > 0.f) kl += qr * (logf(qr) - (lr - ls));
        g.kl[t] = kl;
        if (g.ce) g.ce[t] = !has_label ? 0.f : u.s == 0.f ? -ninf() : l1 - (z_label - m);
        if (g.stats) {
          g.stats[4 * t] = m;
          g.stats[4 * t + 1] = ls;
          g.stats[4 * t + 2] = lr;
          g.stats[4 * t + 3] = l1;
        }
      }
    }
  }
  if constexpr (kMode != 0) {
    T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
    const bool vec = misaligned(out) == a;
    const bool none = m == ninf();
    const float w = g.dkl ? g.dkl[t] / tau : 0.f;
    const float w1 = (g.dce && has_label) ? g.dce[t] : 0.f;
    // a bucket in which the student can have nothing is dropped
    const float q_rest = lr == ninf() ? 0.f : sh.q_rest;
    const float q_all = sh.q_sum + q_rest;
    // p's factor off the list
    const float wp = w * (q_rest > 0.f ? q_all - q_rest / expf(lr - ls) : q_all);
    const float c1 = 1.f / tau;
    auto grad = [&](float z, float wk) {
      const float d = z - m;
      float y = wk * ex2((d * c1 - ls) * kLog2e);
      if (kTwo) y = fmaf(w1, ex2((d - l1) * kLog2e), y);
      return none ? 0.f : y;
    };
    const float add1 = kTwo ? 0.f : w1;  // one temperature: both softmaxes are the same
    for (int v = tid; v < nvec; v += kThreads) {
      float x[N];
      load_vec(row, v * N - a, V, x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = grad(x[j], wp + add1);
      store_vec(out, v * N - a, V, vec, x);
    }
    __syncthreads();
    // the listed columns and the label get their own terms (this CTA wrote them above)
    if (tid < K && sh.idx[tid] >= 0) {
      float y = grad(sh.z[tid], w * q_all + add1);
      if (!none) y -= w * sh.q[tid] + (sh.idx[tid] == label ? w1 : 0.f);
      out[sh.idx[tid]] = static_cast<T>(y);
    }
    if (tid == K && has_label && !sh.label_listed) {
      const float y = grad(z_label, wp + add1);
      out[label] = static_cast<T>(none ? 0.f : y - w1);
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const p24_logprobs_args& g, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(g.T));
  cudaError_t e;
  if (g.dtype == P24_BF16)
    e = g.entropy ? launch_plain(logprobs_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, s, g)
                  : launch_plain(logprobs_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, g);
  else
    e = g.entropy ? launch_plain(logprobs_kernel<float, true>, grid, dim3(kThreads), 0, s, g)
                  : launch_plain(logprobs_kernel<float, false>, grid, dim3(kThreads), 0, s, g);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_logprobs_bwd(const p24_logprobs_args& g, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(g.T));
  cudaError_t e;
  if (g.dtype == P24_BF16)
    e = g.dentropy ? launch_plain(logprobs_bwd_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, s, g)
                   : launch_plain(logprobs_bwd_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, g);
  else
    e = g.dentropy ? launch_plain(logprobs_bwd_kernel<float, true>, grid, dim3(kThreads), 0, s, g)
                   : launch_plain(logprobs_bwd_kernel<float, false>, grid, dim3(kThreads), 0, s, g);
  if (e == cudaSuccess) count_launch();
  return e;
}

namespace {
template <typename T, bool kTwo, int kMode>
cudaError_t launch_distill_as(const p24_distill_args& g, cudaStream_t s) {
  const size_t smem = (kMode != 2 && (g.flags & P24_DISTILL_TAIL)) ? (g.V / Vec<T>::N + 2 + 15) / 16 * 16 : 0;
  auto kern = distill_kernel<T, kTwo, kMode>;
  if (smem > 32 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_plain(kern, dim3(static_cast<unsigned>(g.T)), dim3(kThreads), smem, s, g);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <int kMode>
cudaError_t launch_distill_mode(const p24_distill_args& g, cudaStream_t s) {
  const bool two = g.labels && g.temperature != 1.f;
  if (g.dtype == P24_BF16)
    return two ? launch_distill_as<__nv_bfloat16, true, kMode>(g, s)
               : launch_distill_as<__nv_bfloat16, false, kMode>(g, s);
  return two ? launch_distill_as<float, true, kMode>(g, s) : launch_distill_as<float, false, kMode>(g, s);
}
}  // namespace

cudaError_t launch_distill(const p24_distill_args& g, cudaStream_t s) {
  return g.dlogits ? launch_distill_mode<1>(g, s) : launch_distill_mode<0>(g, s);
}

cudaError_t launch_distill_bwd(const p24_distill_args& g, cudaStream_t s) { return launch_distill_mode<2>(g, s); }

}  // namespace p24
