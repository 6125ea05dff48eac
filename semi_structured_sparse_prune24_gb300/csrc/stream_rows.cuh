// stream_rows.cuh -- what the kernels on rows of hidden states share (RMS norm, embedding, gradient
// norm): fp32 in pairs, a thread's columns of a row and loads and stores of them (embedding), stores of 8
// neighbouring columns (dequantisation), and reductions over a CTA in a fixed order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "p24_internal.h"
#include "p24_ptx.cuh"

namespace p24 {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// Two fp32 operations in one instruction.
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ Two both(float x) { return two(x, x); }
__device__ __forceinline__ void apart(Two p, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.v)); }
__device__ __forceinline__ Two operator+(Two p, Two q) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(p.v), "l"(q.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two p, Two q) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(p.v), "l"(q.v));
  return r;
}
__device__ __forceinline__ Two fma(Two p, Two q, Two s) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(p.v), "l"(q.v), "l"(s.v));
  return r;
}
// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
};

// Two bf16 of a register as fp32.
__device__ __forceinline__ void widen(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void pack8(Raw8<bf16>& r, const float (&v)[8]) {
  r.q[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void pack8(Raw8<float>& r, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.q[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                        __float_as_uint(v[4 * i + 3]));
}

__device__ __forceinline__ uint32_t bits_of(bf16 x) { return __bfloat16_as_ushort(x); }
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }

// Columns [c, c + 8) of a row of d columns, without those outside it. `vec`: pieces lie on 16-byte boundaries.
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int d, bool vec, const float (&v)[8]) {
  if (vec && c >= 0 && c + 8 <= d) {
    Raw8<T> r;
    pack8(r, v);
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(row + c)[i] = r.q[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i >= 0 && c + i < d) row[c + i] = static_cast<T>(v[i]);
  }
}

// A thread's 8 columns of a row, in pieces of E neighbours that are moved at once, piece p `width` pieces from the one
// before. Where every row of a matrix lies on 16-byte boundaries E is 8, or 4 where a matrix is fp32: then too a warp's
// access covers whole sectors. Other rows take E = 1 for the same reason (16384 x 767 bf16 looked up with 8 neighbours
// an element at a time 36 us, like this 17).
template <int E>
struct Columns {
  int c, step, d;  // the first, from one piece to the next, of a row
  __device__ __forceinline__ Columns(int chunk, int tid, int width, int d_) : c(chunk * width * 8 + E * tid), step(E * width), d(d_) {}
  __device__ __forceinline__ bool none() const { return c >= d; }
};
// E elements in one access.
template <int bytes>
struct Word;
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<32> { struct type { uint4 q[2]; }; };

// A thread's elements as they lie in memory; those outside the row are 0.
template <int E, typename T>
struct Loaded {
  union {
    typename Word<E * sizeof(T)>::type w[8 / E];
    uint32_t u[2 * sizeof(T)];
  };
};
template <typename T>
struct Loaded<1, T> {  // (pairs of bf16 in a register would be put together load by load)
  T e[8];
};
template <int E, typename T>
__device__ __forceinline__ Loaded<E, T> load_columns(const T* row, const Columns<E>& k) {
  Loaded<E, T> x;
  if constexpr (E == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x.e[i] = k.c + i * k.step < k.d ? row[k.c + i * k.step] : static_cast<T>(0.f);
    return x;
  } else {
    using W = typename Word<E * sizeof(T)>::type;
#pragma unroll
    for (unsigned i = 0; i < 2 * sizeof(T); ++i) x.u[i] = 0;
#pragma unroll
    for (int p = 0; p < 8 / E; ++p) {
      const int c = k.c + p * k.step;
      if (c + E <= k.d) {
        x.w[p] = *reinterpret_cast<const W*>(row + c);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (c + i < k.d) {
            const int at = p * E + i;
            if (sizeof(T) == 4) x.u[at] = bits_of(row[c + i]);
            else x.u[at / 2] |= bits_of(row[c + i]) << (16 * (at & 1));
          }
      }
    }
    return x;
  }
}
template <int E, typename T>
__device__ __forceinline__ void values(const Loaded<E, T>& x, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (E == 1) v[i] = to_float(x.e[i]);
    else if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(x.u[i]);
    else if ((i & 1) == 0) widen(x.u[i / 2], v[i], v[i + 1]);
  }
}
template <int E, typename T>
__device__ __forceinline__ void store_columns(T* row, const Columns<E>& k, const float (&v)[8]) {
  if constexpr (E == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k.c + i * k.step < k.d) row[k.c + i * k.step] = static_cast<T>(v[i]);
  } else {
    using W = typename Word<E * sizeof(T)>::type;
    Loaded<E, T> x;
#pragma unroll
    for (unsigned i = 0; i < 2 * sizeof(T); ++i) {
      if constexpr (sizeof(T) == 4) x.u[i] = __float_as_uint(v[i]);
      else x.u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int p = 0; p < 8 / E; ++p) {
      const int c = k.c + p * k.step;
      if (c + E <= k.d) {
        *reinterpret_cast<W*>(row + c) = x.w[p];
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (c + i < k.d) row[c + i] = static_cast<T>(v[p * E + i]);
      }
    }
  }
}

__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
  return x;
}
// The larger of two; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int i = 16; i; i >>= 1) x = max_nan(x, __shfl_xor_sync(~0u, x, i));
  return x;
}

// Sum (or maximum) over a CTA, in every thread, in a fixed order. `part`: shared, 32 floats, not used
// by the reduction before it.
__device__ __forceinline__ float cta_add(float x, float* part) {
  x = warp_add(x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  const unsigned lane = threadIdx.x & 31;
  return warp_add(lane < (blockDim.x >> 5) ? part[lane] : 0.f);
}
__device__ __forceinline__ float cta_max(float x, float* part) {
  x = lanes_max(x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  const unsigned lane = threadIdx.x & 31;
  return lanes_max(lane < (blockDim.x >> 5) ? part[lane] : 0.f);
}

// Threads of a row, 8 columns each: a power of two up to `most`, and chunks of as many.
struct RowThreads {
  int x;
  unsigned chunks;
};
inline RowThreads row_threads(int64_t d, int most) {
  const int64_t n = (d + 7) / 8;
  RowThreads r{32, 1};
  while (r.x < most && r.x < n) r.x *= 2;
  r.chunks = static_cast<unsigned>((n + r.x - 1) / r.x);
  return r;
}
inline bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int size_of(int32_t dtype) { return dtype == P24_BF16 ? 2 : dtype == P24_F32 ? 4 : 1; }
// Whether every row of bf16 or fp32 starts on a 16-byte boundary.
inline bool rows_aligned(const void* p, int64_t ld, int32_t dtype) {
  return !p || ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * size_of(dtype))) & 15u) == 0;
}

}  // namespace
}  // namespace p24
