// norm_kernels.cu -- root-mean-square norm of rows of hidden states with the residual's addition, its
// gradient, and the 8-bit form (e4m3 with a scale for each row or group of columns).
//
//   h = x + r (rounded to r's type),  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w
//   dx = dres + rstd (g - xh mean(g xh)),  g = dy w,  xh = h rstd;   dw = sum over the rows of dy xh
//
// Everything between loads and stores is fp32, the sums in a fixed order; each output is rounded once.
// The bound is memory: a row is read and written once.
#include <algorithm>

#include "stream_rows.cuh"

namespace p24 {
namespace {

constexpr int kWarpPieces = 128;  // rows of up to so many pieces: a warp each

// What the row's lead tensor says about phases: row t's is (first + t step) mod 8.
struct Phase {
  int first, step;
  __device__ __forceinline__ int of(int64_t t) const { return static_cast<int>((first + t * step) & 7); }
};

// The weights of columns [c, c + 8); 1 without weights.
__device__ __forceinline__ void weights8(const void* w, int32_t dtype, int c, int d, bool vec, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  } else if (dtype == P24_BF16) {
    unpack8(load8(static_cast<const bf16*>(w), c, d, vec), v);
  } else {
    unpack8(load8(static_cast<const float*>(w), c, d, vec), v);
  }
}

__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ void store_e4m3(uint8_t* row, int c, int d, bool vec, const float (&v)[8]) {
  const uint2 q = e4m3x8(v);
  if (vec && c >= 0 && c + 8 <= d) {
    *reinterpret_cast<uint2*>(row + c) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i >= 0 && c + i < d) row[c + i] = static_cast<uint8_t>((i < 4 ? q.x >> (8 * i) : q.y >> (8 * (i - 4))) & 255u);
  }
}

// A scale and what values are multiplied by, from the largest magnitude. The reciprocal is that of the
// stored scale, so that code times scale is the nearest to the value that the code allows; below 2^-118
// a scale's reciprocal leaves fp32's range, and the scale stays there.
__device__ __forceinline__ float scale_of(float top) { return top == 0.f ? 1.f : max_nan(top * (1.f / 448.f), 0x1p-118f); }

// kWarp: a warp takes a row, else the CTA. NV: pieces of a thread.
template <typename Tx, typename Tr, bool kWarp, bool kAligned, int NV>
__global__ void __launch_bounds__(kWarp ? 256 : 1024) rmsnorm_kernel(const p24_rmsnorm_args g, const Phase phase) {
  __shared__ float part[4][32];
  extern __shared__ float group_top[];  // 8 bits, phases: the groups' largest magnitudes
  const int d = static_cast<int>(g.d), lane = threadIdx.x & 31;
  const int tid = kWarp ? lane : threadIdx.x, NT = kWarp ? 32 : blockDim.x;
  const int per = kWarp ? blockDim.x >> 5 : 1;
  int64_t t = static_cast<int64_t>(blockIdx.x) * per + (kWarp ? threadIdx.x >> 5 : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  const bool quant = g.y_dtype == P24_E4M3;
  const int groups = quant ? (d + g.group - 1) / g.group : 0;
  float* tops = group_top + (kWarp ? (threadIdx.x >> 5) * groups : 0);
  auto add = [&](float x, int k) { return kWarp ? warp_add(x) : cta_add(x, part[k]); };
  auto join = [&] {
    if (kWarp) __syncwarp(); else __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  for (; t < g.T; t += step) {
    const int s = kAligned ? 0 : phase.of(t);
    const int n = (d + s + 7) >> 3;
    const Tx* x = static_cast<const Tx*>(g.x) + t * g.ldx;
    const Tr* r = static_cast<const Tr*>(g.r) + (g.r ? t * g.ldr : 0);
    const bool xv = kAligned || pieces_aligned(x, s), rv = kAligned || pieces_aligned(r, s);
    Raw8<Tx> rx[NV];
    Raw8<Tr> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid;
      if (j < n) rx[i] = load8(x, 8 * j - s, d, xv);
    }
    if (g.r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * NT + tid;
        if (j < n) rr[i] = load8(r, 8 * j - s, d, rv);
      }
    }
    float h[NV][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = 0.f;
      if (j < n) {
        unpack8(rx[i], h[i]);
        if (g.r) {
          float b[8];
          unpack8(rr[i], b);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][k] = to_float(static_cast<Tr>(h[i][k] + b[k]));
          Tr* to = static_cast<Tr*>(g.h) + t * g.ldh;
          store8(to, 8 * j - s, d, kAligned || pieces_aligned(to, s), h[i]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(h[i][k], h[i][k], sum);
    }
    sum = add(sum, 0);
    float rstd = rsqrtf(sum / static_cast<float>(d) + g.eps);
    if (sum == __int_as_float(0x7f800000)) {  // squares beyond fp32 (or an infinity): at a scale of 2^-80
      float small = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) small = fmaf(h[i][k] * 0x1p-80f, h[i][k] * 0x1p-80f, small);
      small = add(small, 1);
      rstd = 0x1p-80f * rsqrtf(small / static_cast<float>(d));
    }
    if (g.rstd && tid == 0) g.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid;
      if (j < n) {
        float w[8];
        weights8(g.w, g.w_dtype, 8 * j - s, d, kAligned, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] = h[i][k] * rstd * w[k];
      }
    }
    if (!quant) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * NT + tid, c = 8 * j - s;
        if (j >= n) continue;
        if (g.y_dtype == P24_BF16) {
          bf16* y = static_cast<bf16*>(g.y) + t * g.ldy;
          store8(y, c, d, kAligned || pieces_aligned(y, s), h[i]);
        } else {
          float* y = static_cast<float*>(g.y) + t * g.ldy;
          store8(y, c, d, kAligned || pieces_aligned(y, s), h[i]);
        }
      }
    } else {
      uint8_t* y = static_cast<uint8_t*>(g.y) + t * g.ldy;
      const bool yv = kAligned || (reinterpret_cast<uintptr_t>(y + 8 - s) & 7u) == 0;
      float* scales = g.scale + t * g.lds;
      if (groups == 1) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(h[i][k]));
        const float sc = scale_of(kWarp ? lanes_max(top) : cta_max(top, part[2]));
        if (tid == 0) scales[0] = sc;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int j = i * NT + tid;
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][k] *= 1.f / sc;
          if (j < n) store_e4m3(y, 8 * j - s, d, yv, h[i]);
        }
      } else {
        // A piece of 8 columns meets at most two groups. Magnitudes are ordered as whole numbers, NaN last.
        for (int i = tid; i < groups; i += NT) tops[i] = 0.f;
        join();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int j = i * NT + tid, c = 8 * j - s;
          if (j >= n) continue;
          const int a = max(c, 0) / g.group, b = min(c + 7, d - 1) / g.group;
          float ta = 0.f, tb = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float m = fabsf(h[i][k]);
            if (c + k < b * g.group || a == b) ta = max_nan(ta, m); else tb = max_nan(tb, m);
          }
          atomicMax(reinterpret_cast<int*>(&tops[a]), __float_as_int(ta));
          if (a != b) atomicMax(reinterpret_cast<int*>(&tops[b]), __float_as_int(tb));
        }
        join();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int j = i * NT + tid, c = 8 * j - s;
          if (j >= n) continue;
          const int a = max(c, 0) / g.group, b = min(c + 7, d - 1) / g.group;
          const float ia = 1.f / scale_of(tops[a]), ib = 1.f / scale_of(tops[b]);
#pragma unroll
          for (int k = 0; k < 8; ++k) h[i][k] *= (c + k < b * g.group || a == b) ? ia : ib;
          store_e4m3(y, c, d, yv, h[i]);
        }
        for (int i = tid; i < groups; i += NT) scales[i] = scale_of(tops[i]);
      }
    }
    join();  // before the next row's reductions write again
  }
}

// The gradient. The weight's is summed over the rows of a CTA in registers where a thread's columns are
// the same in every row (kAligned), else in shared memory, and goes to the CTA's row of `parts`.
template <typename Th, typename Td, bool kAligned, int NV>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_kernel(const p24_rmsnorm_bwd_args g, const Phase phase, float* parts) {
  __shared__ float part[2][32];
  extern __shared__ float dw_sh[];
  const int d = static_cast<int>(g.d), tid = threadIdx.x, NT = blockDim.x;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.f;
  if (!kAligned && parts)
    for (int c = tid; c < d; c += NT) dw_sh[c] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  int odd = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x, odd ^= 1) {
    const int s = kAligned ? 0 : phase.of(t);
    const int n = (d + s + 7) >> 3;
    const Th* h = static_cast<const Th*>(g.h) + t * g.ldh;
    const Td* dy = static_cast<const Td*>(g.dy) + t * g.lddy;
    const bool hv = kAligned || pieces_aligned(h, s), dv = kAligned || pieces_aligned(dy, s);
    const float rstd = g.rstd[t];
    Raw8<Th> rh[NV];
    Raw8<Td> rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid;
      if (j < n) rh[i] = load8(h, 8 * j - s, d, hv), rd[i] = load8(dy, 8 * j - s, d, dv);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid, c = 8 * j - s;
      if (j >= n) continue;
      float xh[8], v[8], w[8];
      unpack8(rh[i], xh);
      unpack8(rd[i], v);
      weights8(g.w, g.w_dtype, c, d, kAligned, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float p = v[k] * (xh[k] * rstd);
        sum = fmaf(p, w[k], sum);
        if (kAligned) acc[i][k] += p;
        else if (parts && c + k >= 0 && c + k < d) dw_sh[c + k] += p;
      }
    }
    const float mean = cta_add(sum, part[odd]) / static_cast<float>(d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * NT + tid, c = 8 * j - s;
      if (j >= n) continue;
      float xh[8], v[8], w[8];
      unpack8(rh[i], xh);
      unpack8(rd[i], v);
      weights8(g.w, g.w_dtype, c, d, kAligned, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = rstd * (v[k] * w[k] - xh[k] * rstd * mean);
      if (g.dres) {
        if (g.r_dtype == P24_BF16) {
          const bf16* r = static_cast<const bf16*>(g.dres) + t * g.ldres;
          unpack8(load8(r, c, d, kAligned || pieces_aligned(r, s)), w);
        } else {
          const float* r = static_cast<const float*>(g.dres) + t * g.ldres;
          unpack8(load8(r, c, d, kAligned || pieces_aligned(r, s)), w);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += w[k];
      }
      if (g.dx_dtype == P24_BF16) {
        bf16* to = static_cast<bf16*>(g.dx) + t * g.lddx;
        store8(to, c, d, kAligned || pieces_aligned(to, s), v);
      } else {
        float* to = static_cast<float*>(g.dx) + t * g.lddx;
        store8(to, c, d, kAligned || pieces_aligned(to, s), v);
      }
    }
    // the next row's phase gives a column to another thread
    if (!kAligned) __syncthreads();
  }
  if (!parts) return;
  float* to = parts + static_cast<int64_t>(blockIdx.x) * d;
  if (kAligned) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * NT + tid);
      if (c < d) store8(to, c, d, (d & 3) == 0, acc[i]);
    }
  } else {
    for (int c = tid; c < d; c += NT) to[c] = dw_sh[c];
  }
}

// Column sums of the CTAs' parts [G, d]: 32 columns of a CTA, 8 warps that take every eighth row.
__global__ void __launch_bounds__(256) dweight_kernel(const float* parts, int G, int d, float* dw) {
  __shared__ float sh[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = warp; i < G; i += 8) s += parts[static_cast<int64_t>(i) * d + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sh[i][lane];
    dw[c] = s;
  }
}

// Values of 8-bit codes: a thread takes 8 columns.
template <typename To>
__global__ void __launch_bounds__(256) dequant8_kernel(const p24_dequant8_args g, bool qv, bool yv) {
  const int d = static_cast<int>(g.d), n = (d + 7) >> 3;
  const int64_t all = g.T * n;
  pdl_wait();
  pdl_trigger();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / n;
    const int c = static_cast<int>(i - t * n) * 8;
    const uint8_t* q = static_cast<const uint8_t*>(g.q) + t * g.ldq;
    uint2 b = make_uint2(0, 0);
    if (qv && c + 8 <= d) {
      b = *reinterpret_cast<const uint2*>(q + c);
    } else {
      for (int k = 0; k < 8; ++k)
        if (c + k < d) (k < 4 ? b.x : b.y) |= static_cast<uint32_t>(q[c + k]) << (8 * (k & 3));
    }
    const float sc = g.scale[t * g.lds + c / g.group];
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((k < 2 ? b.x : b.y) >> (16 * (k & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * k] = f.x * sc;
      v[2 * k + 1] = f.y * sc;
    }
    store8(static_cast<To*>(g.y) + t * g.ldy, c, d, yv, v);
  }
}

template <typename Tx, typename Tr, bool kWarp, bool kAligned>
cudaError_t launch_norm_as(const p24_rmsnorm_args& g, Phase ph, int pieces, cudaStream_t s) {
  const int groups = g.y_dtype == P24_E4M3 ? static_cast<int>((g.d + g.group - 1) / g.group) : 0;
  auto go = [&](auto kern, int nv) {
    const int NT = kWarp ? 256 : ((pieces + nv - 1) / nv + 31) / 32 * 32;
    const size_t smem = groups > 1 ? groups * sizeof(float) * (kWarp ? NT / 32 : 1) : 0;
    const int64_t rows = kWarp ? (g.T + NT / 32 - 1) / (NT / 32) : g.T;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(std::min<int64_t>(rows, sm_count() * 16))), dim3(NT), smem, s, g, ph);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (kWarp) {
    if (pieces <= 32) return go(rmsnorm_kernel<Tx, Tr, true, kAligned, 1>, 1);
    return go(rmsnorm_kernel<Tx, Tr, true, kAligned, 4>, 4);
  }
  if (pieces <= 1024 && (g.T <= 2 * sm_count() || pieces <= 256)) return go(rmsnorm_kernel<Tx, Tr, false, kAligned, 1>, 1);
  if (pieces <= 1024) return go(rmsnorm_kernel<Tx, Tr, false, kAligned, 2>, 2);
  return go(rmsnorm_kernel<Tx, Tr, false, kAligned, 5>, 5);
}
template <typename Tx, typename Tr>
cudaError_t launch_norm_types(const p24_rmsnorm_args& g, Phase ph, bool aligned, cudaStream_t s) {
  const int pieces = static_cast<int>((g.d + (aligned ? 0 : 7) + 7) / 8);
  if (pieces <= kWarpPieces)
    return aligned ? launch_norm_as<Tx, Tr, true, true>(g, ph, pieces, s) : launch_norm_as<Tx, Tr, true, false>(g, ph, pieces, s);
  return aligned ? launch_norm_as<Tx, Tr, false, true>(g, ph, pieces, s) : launch_norm_as<Tx, Tr, false, false>(g, ph, pieces, s);
}

// The phase of the first bf16 tensor among these, which fp32 ones of the same layout agree with.
struct Lead {
  const void* p;
  int64_t ld;
  int32_t dtype;
};
Phase phase_of(std::initializer_list<Lead> all) {
  const Lead* lead = all.begin();
  for (const Lead& l : all)
    if (l.p && l.dtype == P24_BF16) {
      lead = &l;
      break;
    }
  const uintptr_t at = reinterpret_cast<uintptr_t>(lead->p) / size_of(lead->dtype);
  return Phase{static_cast<int>(at & 7), static_cast<int>(lead->ld & 7)};
}

// CTAs of the gradient, each with a row of partial sums: 2 for each SM.
int64_t bwd_ctas(int64_t T) { return std::min<int64_t>(T, 2 * sm_count()); }

template <typename Th, typename Td, bool kAligned>
cudaError_t launch_bwd_as(const p24_rmsnorm_bwd_args& g, Phase ph, float* parts, cudaStream_t s) {
  const int pieces = static_cast<int>((g.d + (kAligned ? 0 : 7) + 7) / 8);
  auto go = [&](auto kern, int nv) {
    const int NT = ((pieces + nv - 1) / nv + 31) / 32 * 32;
    const size_t smem = kAligned || !parts ? 0 : g.d * sizeof(float);
    if (smem > 40 << 10) {
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
      if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(bwd_ctas(g.T))), dim3(NT), smem, s, g, ph, parts);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (pieces <= 512) return go(rmsnorm_bwd_kernel<Th, Td, kAligned, 1>, 1);
  if (pieces <= 2048) return go(rmsnorm_bwd_kernel<Th, Td, kAligned, 2>, 2);
  return go(rmsnorm_bwd_kernel<Th, Td, kAligned, 5>, 5);
}
template <typename Th, typename Td>
cudaError_t launch_bwd_types(const p24_rmsnorm_bwd_args& g, Phase ph, bool aligned, float* parts, cudaStream_t s) {
  return aligned ? launch_bwd_as<Th, Td, true>(g, ph, parts, s) : launch_bwd_as<Th, Td, false>(g, ph, parts, s);
}

}  // namespace

int64_t rmsnorm_bwd_parts(int64_t T, int64_t d) { return bwd_ctas(T) * d; }

cudaError_t launch_rmsnorm(const p24_rmsnorm_args& a, cudaStream_t s) {
  p24_rmsnorm_args g = a;
  if (!g.r) g.r_dtype = g.x_dtype, g.h = nullptr;
  if (g.y_dtype == P24_E4M3 && (g.group == 0 || g.group > g.d)) g.group = static_cast<int32_t>(g.d);
  const bool aligned = rows_aligned(g.x, g.ldx, g.x_dtype) && rows_aligned(g.r, g.ldr, g.r_dtype) && on16(g.w) &&
                       rows_aligned(g.h, g.ldh, g.r_dtype) && rows_aligned(g.y, g.ldy, g.y_dtype);
  const Phase ph = phase_of({{g.x, g.ldx, g.x_dtype}, {g.y, g.ldy, g.y_dtype}, {g.r, g.ldr, g.r_dtype}});
  if (g.x_dtype == P24_BF16)
    return g.r_dtype == P24_BF16 ? launch_norm_types<bf16, bf16>(g, ph, aligned, s) : launch_norm_types<bf16, float>(g, ph, aligned, s);
  return g.r_dtype == P24_BF16 ? launch_norm_types<float, bf16>(g, ph, aligned, s) : launch_norm_types<float, float>(g, ph, aligned, s);
}

cudaError_t launch_rmsnorm_bwd(const p24_rmsnorm_bwd_args& g, float* parts, cudaStream_t s) {
  const bool aligned = rows_aligned(g.h, g.ldh, g.h_dtype) && rows_aligned(g.dy, g.lddy, g.dy_dtype) && on16(g.w) &&
                       rows_aligned(g.dres, g.ldres, g.r_dtype) && rows_aligned(g.dx, g.lddx, g.dx_dtype);
  const Phase ph = phase_of({{g.h, g.ldh, g.h_dtype}, {g.dy, g.lddy, g.dy_dtype}, {g.dx, g.lddx, g.dx_dtype}, {g.dres, g.ldres, g.r_dtype}});
  float* to = g.dw ? parts : nullptr;
  cudaError_t e;
  if (g.h_dtype == P24_BF16)
    e = g.dy_dtype == P24_BF16 ? launch_bwd_types<bf16, bf16>(g, ph, aligned, to, s) : launch_bwd_types<bf16, float>(g, ph, aligned, to, s);
  else
    e = g.dy_dtype == P24_BF16 ? launch_bwd_types<float, bf16>(g, ph, aligned, to, s) : launch_bwd_types<float, float>(g, ph, aligned, to, s);
  if (e != cudaSuccess || !g.dw) return e;
  const int d = static_cast<int>(g.d);
  e = launch_pdl(dweight_kernel, dim3((d + 31) / 32), dim3(256), 0, s, static_cast<const float*>(parts), static_cast<int>(bwd_ctas(g.T)), d, g.dw);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_dequant8(const p24_dequant8_args& a, cudaStream_t s) {
  p24_dequant8_args g = a;
  if (g.group == 0 || g.group > g.d) g.group = static_cast<int32_t>(g.d);
  const bool qv = rows_aligned(g.q, g.ldq, P24_E4M3), yv = rows_aligned(g.y, g.ldy, g.y_dtype);
  const int64_t blocks = std::min<int64_t>((g.T * ((g.d + 7) / 8) + 255) / 256, sm_count() * 64);
  const cudaError_t e = g.y_dtype == P24_BF16
                            ? launch_pdl(dequant8_kernel<bf16>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, g, qv, yv)
                            : launch_pdl(dequant8_kernel<float>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, g, qv, yv);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace p24
