// norm_kernels.cu -- root-mean-square norm of rows of hidden states with the residual's addition, its
// gradient, and the 8-bit form (e4m3 with a scale for each row or group of columns).
//
//   h = x + r (rounded to r's type),  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w
//   dx = dres + rstd (g - xh mean(g xh)),  g = dy w,  xh = h rstd;   dw = sum over the rows of dy xh
//
// Everything between loads and stores is fp32, the sums in a fixed order; each output is rounded once.
// The bound is memory: a row is read and written once. 16384 x 8192 bf16 with the residual's addition takes 168 us
// (6.4 TB/s), the gradient with the skip connection's 158 (6.8).
//
// A unit (a CTA, or a warp for rows of up to 512 columns) takes rows unit, unit + units, ... A row is its interior,
// from a boundary of 8 elements to another, and at most 7 edge columns before and after it. The interior is cut into
// pieces of E columns, thread i has pieces i, i + NT, ...; edge columns are single threads'. E is 8 where all
// matrices are bf16, else 4: then 16 bytes of fp32 and 8 of bf16 are neighbouring threads' neighbours (with pieces of
// 8 columns a warp's access to fp32 touched each sector twice: norm of 16384 x 8192 fp32 428 us against 322).
// The interiors of the rows ahead come by bulk copies into a ring of S rows in the unit's shared memory, and go on
// arriving through a row's reduction and its stores. Copies by each thread into slots of its own (cp.async) took
// 65 more of 260 instructions a warp and piece, and in rows that start 16 bytes off a sector 1.6 times the L2
// reads: the gradient of 16384 x 8191 252 us against 200.
#include <algorithm>
#include <type_traits>

#include "stream_rows.cuh"

namespace p24 {
namespace {

// What the rows' lead tensor says about phases: row t starts (first + t step) mod 8 elements past a boundary. Units
// are as many as a multiple of 8 (or no fewer than rows), so that all rows of a unit have one phase.
struct Phase {
  int first, step;
  __device__ __forceinline__ int of(int64_t t) const { return static_cast<int>((first + t * step) & 7); }
};

// A matrix that rows come from or go to, bf16 or fp32 (f32: 0 or 1).
struct Matrix {
  uint8_t* p;
  int64_t ld;  // bytes
  int f32;
  __device__ __forceinline__ Matrix() {}
  __device__ __forceinline__ Matrix(const void* q, int64_t elements, int32_t dtype)
      : p(static_cast<uint8_t*>(const_cast<void*>(q))), ld(elements << (1 + (dtype == P24_F32))), f32(dtype == P24_F32) {}
  __device__ __forceinline__ uint8_t* row(int64_t t) const { return p + t * ld; }
};

// E columns of a row as fp32 pairs.
template <int E>
struct Vals {
  Two p[E / 2];
};
template <int E>
__device__ __forceinline__ void to_array(const Vals<E>& a, float (&v)[E]) {
#pragma unroll
  for (int k = 0; k < E / 2; ++k) apart(a.p[k], v[2 * k], v[2 * k + 1]);
}
template <int E>
__device__ __forceinline__ Vals<E> filled(float x) {
  Vals<E> a;
#pragma unroll
  for (int k = 0; k < E / 2; ++k) a.p[k] = both(x);
  return a;
}
template <int E>
__device__ __forceinline__ float sum_of(const Two& t) {
  float a, b;
  apart(t, a, b);
  return a + b;
}
__device__ __forceinline__ Two pair_of(uint32_t w) { return two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ float rounded_bf16(float x) { return to_float(static_cast<bf16>(x)); }

// A piece: of 8 bf16 (16 bytes), of 4 bf16 (8 bytes), of 4 fp32 (16 bytes).
__device__ __forceinline__ Vals<8> vals_of(const uint4& q) {
  Vals<8> a;
  a.p[0] = pair_of(q.x), a.p[1] = pair_of(q.y), a.p[2] = pair_of(q.z), a.p[3] = pair_of(q.w);
  return a;
}
__device__ __forceinline__ Vals<4> vals_of(const uint2& q) {
  Vals<4> a;
  a.p[0] = pair_of(q.x), a.p[1] = pair_of(q.y);
  return a;
}
__device__ __forceinline__ Vals<4> vals_of_f32(const uint4& q) {
  Vals<4> a;
  a.p[0] = two(__uint_as_float(q.x), __uint_as_float(q.y)), a.p[1] = two(__uint_as_float(q.z), __uint_as_float(q.w));
  return a;
}
__device__ __forceinline__ float element(const uint8_t* row, int f32, int c) {
  return f32 ? reinterpret_cast<const float*>(row)[c] : to_float(reinterpret_cast<const bf16*>(row)[c]);
}
__device__ __forceinline__ void put_element(uint8_t* row, int f32, int c, float x) {
  if (f32) reinterpret_cast<float*>(row)[c] = x;
  else reinterpret_cast<bf16*>(row)[c] = static_cast<bf16>(x);
}
// Columns [c, c + E) of a row; `vec`: in one access.
template <int E>
__device__ __forceinline__ Vals<E> load_vals(const uint8_t* row, int f32, int c, bool vec) {
  if (vec) {
    if constexpr (E == 8) {
      if (!f32) return vals_of(*reinterpret_cast<const uint4*>(row + 2 * c));
      const Vals<4> a = vals_of_f32(*reinterpret_cast<const uint4*>(row + 4 * c)), b = vals_of_f32(*reinterpret_cast<const uint4*>(row + 4 * c + 16));
      return Vals<8>{{a.p[0], a.p[1], b.p[0], b.p[1]}};
    } else if (f32) return vals_of_f32(*reinterpret_cast<const uint4*>(row + 4 * c));
    else return vals_of(*reinterpret_cast<const uint2*>(row + 2 * c));
  }
  Vals<E> a;
#pragma unroll
  for (int k = 0; k < E / 2; ++k) a.p[k] = two(element(row, f32, c + 2 * k), element(row, f32, c + 2 * k + 1));
  return a;
}
template <int E>
__device__ __forceinline__ void store_vals(uint8_t* row, int f32, int c, bool vec, const Vals<E>& a) {
  float v[E];
  to_array(a, v);
  if (vec) {
    if constexpr (E == 8) {
      *reinterpret_cast<uint4*>(row + 2 * c) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else if (f32) {
      *reinterpret_cast<float4*>(row + 4 * c) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(row + 2 * c) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) put_element(row, f32, c + k, v[k]);
  }
}

__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
// One of the arrivals that `bar` counts, once this thread's copy4s so far are there.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t shared4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 shared8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// How a row is split over a unit's threads, the same for all rows of the unit.
template <int E, bool kAligned>
struct Split {
  int NT, tid, d, c0, n, edges, edge;  // c0: the interior's first column; n pieces; this thread's edge column, if any
  __device__ __forceinline__ void start(int phase) {
    c0 = kAligned ? 0 : min(-phase & 7, d);
    n = (d - c0) / 8 * (8 / E);
    edges = kAligned ? 0 : d - n * E;
    edge = tid < c0 ? tid : n * E + tid;
  }
  __device__ __forceinline__ bool has(int i) const { return i * NT + tid < n; }
  __device__ __forceinline__ int column(int i) const { return c0 + E * (i * NT + tid); }
  __device__ __forceinline__ bool has_edge() const { return !kAligned && tid < edges; }
  // Whether the pieces of a matrix lie on boundaries of their own size.
  __device__ __forceinline__ bool fits(const Matrix& m, int64_t t) const {
    return kAligned || (reinterpret_cast<uintptr_t>(m.row(t) + (c0 << (m.f32 + 1))) & (E * 2 * (m.f32 + 1) - 1)) == 0;
  }
};

constexpr int kMostRows = 4;  // of a ring

constexpr int kMostEdges = 16;  // 14 are

// What comes beside the interiors of a ring's rows.
template <int M>
struct Beside {
  uint64_t full[kMostRows];  // a row has arrived
  uint32_t edge[kMostRows][M][kMostEdges];
  float rstd[kMostRows];
  int abort;
};

// A unit's rows of M matrices: through a ring of S rows (kRing), or read where they are used. Edge columns, and the
// row's rstd where it is an input, come by copies of 4 bytes, as far ahead as the interiors: loads into registers
// one row ahead were waited for in every row (the gradient of 16384 x 8192 166 us against 158). The word of a bf16
// column has a neighbour in it; where that lies outside the matrix the column is loaded by itself.
template <int M, int NV, int E, bool kAligned, bool kRing>
struct Pieces {
  Split<E, kAligned> sp;
  Matrix in[M];
  int m, row_bytes, S;  // matrices; of a row in the ring; rows of it
  uint32_t base;        // the ring
  int64_t T;
  Beside<M>* sh;
  const float* rstd;    // or null
  int* status;
  int high;             // a bf16 edge column is the upper half of its word
  bool vec[M];
  int stage, parity;    // the row in use

  __device__ __forceinline__ int f32(int a) const { return E == 8 ? 0 : in[a].f32; }
  __device__ __forceinline__ int at(int a) const {  // matrix a's offset in a row of the ring
    int k = 0;
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (i < a && i < m) k += sp.NT * NV * E * 2 << f32(i);
    return k;
  }
  // All threads of the unit; the caller's barrier comes after it and before the first fill.
  __device__ __forceinline__ void start(int64_t t, int phase, const void* smem) {
    sp.start(phase);
    row_bytes = at(M);
    base = smem_u32(smem);
    stage = parity = 0;
    if (!kRing) {
#pragma unroll
      for (int a = 0; a < M; ++a) vec[a] = a < m && sp.fits(in[a], t);
    } else if (sp.tid == 0) {
      sh->abort = 0;
      for (int k = 0; k < S; ++k) mbar_init(&sh->full[k], 1 + feeders());
      fence_barrier_init();
      fence_proxy_async_smem();
    }
    high = (phase + sp.edge) & 1;
  }
  __device__ __forceinline__ int feeders() const { return max(sp.edges, 1); }
  // Threads below feeders(): row t, if there is one, into `to`, which no thread reads any more.
  __device__ __forceinline__ void fill(int64_t t, int to) const {
    if (t >= T || sp.tid >= feeders()) return;
    if (sp.tid == 0) {
      uint32_t bytes = 0;
#pragma unroll
      for (int a = 0; a < M; ++a)
        if (a < m) bytes += sp.n * E * 2 << f32(a);
      mbar_arrive_expect_tx(&sh->full[to], bytes);
      if (sp.n > 0) {
#pragma unroll
        for (int a = 0; a < M; ++a)
          if (a < m) bulk_copy(base + to * row_bytes + at(a), in[a].row(t) + (sp.c0 << (f32(a) + 1)), sp.n * E * 2 << f32(a), &sh->full[to]);
      }
      if (rstd) copy4(smem_u32(&sh->rstd[to]), rstd + t);
    }
    if (sp.has_edge()) {
#pragma unroll
      for (int a = 0; a < M; ++a) {
        if (a >= m) continue;
        const uint8_t* row = in[a].row(t);
        const bool alone = high ? sp.edge == 0 && t == 0 : sp.edge == sp.d - 1 && t == T - 1;
        uint32_t* slot = &sh->edge[to][a][sp.tid];
        if (f32(a)) copy4(smem_u32(slot), row + 4 * sp.edge);
        else if (!alone) copy4(smem_u32(slot), row + 2 * (sp.edge - high));
        else *slot = reinterpret_cast<const uint16_t*>(row)[sp.edge] << (16 * high);
      }
    }
    arrive_after_copies(&sh->full[to]);
  }
  __device__ __forceinline__ void wait() const { p24_wait(&sh->full[stage], parity, &sh->abort, status); }
  __device__ __forceinline__ void advance() {
    if (++stage == S) stage = 0, parity ^= 1;
  }
  // After an expired wait: the last of the unit's rows may still be on their way here.
  __device__ __forceinline__ void drain(int64_t rows) const {
    if (*reinterpret_cast<volatile int*>(&sh->abort) == 0) return;
    for (int64_t i = rows > S ? rows - S : 0; i < rows; ++i) p24_wait_quiet(&sh->full[i % S], (i / S) & 1);
  }
  __device__ __forceinline__ Vals<E> get(int a, int i, int64_t t) const {
    if (!kRing) return load_vals<E>(in[a].row(t), f32(a), sp.column(i), vec[a]);
    const uint32_t from = base + stage * row_bytes + at(a) + ((i * sp.NT + sp.tid) * E * 2 << f32(a));
    if constexpr (E == 8) return vals_of(shared16(from));
    else if (f32(a)) return vals_of_f32(shared16(from));
    else return vals_of(shared8(from));
  }
  // This thread's edge column of the row in use.
  __device__ __forceinline__ float edge(int a, int64_t t) const {
    if (!kRing) return element(in[a].row(t), f32(a), sp.edge);
    const uint32_t w = shared4(smem_u32(&sh->edge[stage][a][sp.tid]));
    return __uint_as_float(f32(a) || high ? (f32(a) ? w : w & 0xffff0000u) : w << 16);
  }
};

// The weights of a thread's columns: in registers, or in shared memory where it has 16 columns, or read each time.
template <int NV, int E>
struct Weights {
  static constexpr int kHow = NV * E <= 8 ? 0 : NV * E <= 16 ? 1 : 2;
  const uint8_t* w;
  int f32;
  bool vec;
  uint32_t sh;
  Vals<E> r[kHow == 0 ? NV : 1];
  float edge;

  template <typename S>
  __device__ __forceinline__ Vals<E> read(const S& sp, int i) const {
    return w ? load_vals<E>(w, f32, sp.column(i), vec) : filled<E>(1.f);
  }
  // smem: the unit's place for them (16 bytes of each thread side by side)
  template <typename S>
  __device__ __forceinline__ void start(const S& sp, const void* weight, int32_t dtype, const void* smem) {
    w = static_cast<const uint8_t*>(weight), f32 = dtype == P24_F32;
    vec = w && (reinterpret_cast<uintptr_t>(w + (sp.c0 << (f32 + 1))) & (E == 4 && !f32 ? 7 : 15)) == 0;
    sh = smem_u32(smem) + 16 * sp.tid;
    edge = sp.has_edge() && w ? element(w, f32, sp.edge) : 1.f;
    if (kHow == 2) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!sp.has(i)) continue;
      const Vals<E> v = read(sp, i);
      if (kHow == 0) {
        r[i] = v;
      } else {
        float x[E];
        to_array(v, x);
#pragma unroll
        for (int k = 0; k < E; k += 4)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sh + (i * E + k) / 4 * 16 * sp.NT), "f"(x[k]), "f"(x[k + 1]),
                       "f"(x[k + 2]), "f"(x[k + 3])
                       : "memory");
      }
    }
  }
  template <typename S>
  __device__ __forceinline__ Vals<E> get(const S& sp, int i) const {
    if (kHow == 0) return r[i];
    if (kHow == 2) return read(sp, i);
    Vals<E> v;
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      const Vals<4> q = vals_of_f32(shared16(sh + (i * E + k) / 4 * 16 * sp.NT));
      v.p[k / 2] = q.p[0], v.p[k / 2 + 1] = q.p[1];
    }
    return v;
  }
};

// Column c of a row of sums in shared memory, one word in nine left out: the lanes of a warp, 8 columns apart,
// meet no conflicts.
__device__ __forceinline__ int padded(int c) { return c + (c >> 3); }

// Codes of 8 bits.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
}
// A scale from the largest magnitude: its product with fp32's 1/448, two units in the last place from the quotient at most
// (any scale near it would do: codes are those of the quotients by the stored one), and no less than 2^-118, below which
// its reciprocal leaves fp32's range.
__device__ __forceinline__ float scale_of(float top) { return top == 0.f ? 1.f : max_nan(top * (1.f / 448.f), 0x1p-118f); }
// What values are divided by, a scale. A quotient is the value times an approximate reciprocal (2 units in the last place
// off at most, the product then 5), and a step of refinement: the remainder is off by 2^-21 of such a unit and its product with
// the reciprocal by 2^-20, so what is rounded in the end is within 2^-19 units of the true quotient. Where that is the
// midpoint of two codes, a number of few bits, the rounding gives exactly it. (The product alone gives one of a midpoint's
// neighbours as often as not; with it 16384 x 4096 bf16 took 53 us with a row's scale, like this 59.) Values come with their
// sign turned, which keeps that of zeros. Beside a scale below 2^-90 the remainder would lie among the smallest numbers: both
// are taken times 2^64. An infinite scale gives 0, and for infinite values NaN; so does a scale that is NaN.
struct Divisor {
  float s, neg, up;  // the scale, which the remainder is found with; -1 / scale; 2^64 or 1
};
__device__ __forceinline__ Divisor by(float scale) {
  Divisor v;
  v.up = scale < 0x1p-90f ? 0x1p64f : 1.f;
  v.s = scale * v.up;
  v.neg = -__fdividef(1.f, v.s);
  if (v.s == __int_as_float(0x7f800000)) v.s = 0.f;
  return v;
}
__device__ __forceinline__ float quotient(float minus, const Divisor& v) {
  minus *= v.up;
  const float q = minus * v.neg;
  return fmaf(fmaf(q, v.s, minus), v.neg, q);
}
// Of -a, the columns from `cut` on by another scale than those before it.
template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int c, bool vec, Vals<E> a, const Divisor& x, const Divisor& y, int cut) {
  float v[E];
  if (x.up != 1.f || y.up != 1.f) {
#pragma unroll
    for (int k = 0; k < E / 2; ++k) a.p[k] = a.p[k] * two(2 * k < cut ? x.up : y.up, 2 * k + 1 < cut ? x.up : y.up);
  }
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const Two s = two(2 * k < cut ? x.s : y.s, 2 * k + 1 < cut ? x.s : y.s), neg = two(2 * k < cut ? x.neg : y.neg, 2 * k + 1 < cut ? x.neg : y.neg);
    const Two q = a.p[k] * neg;
    a.p[k] = fma(fma(q, s, a.p[k]), neg, q);
  }
  to_array(a, v);
  uint32_t q[E / 4];
#pragma unroll
  for (int k = 0; k < E / 4; ++k) q[k] = e4m3x4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  if (vec) {
    if constexpr (E == 8) *reinterpret_cast<uint2*>(row + c) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(row + c) = q[0];
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) row[c + k] = static_cast<uint8_t>(q[k / 4] >> (8 * (k & 3)));
  }
}
template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int c, bool vec, const Vals<E>& a, const Divisor& x) {
  store_e4m3<E>(row, c, vec, a, x, x, E);
}
__device__ __forceinline__ uint8_t e4m3(float x) { return static_cast<uint8_t>(e4m3x4(x, 0.f, 0.f, 0.f)); }
template <int E>
__device__ __forceinline__ float top_of(const Vals<E>& a) {
  float v[E], top = 0.f;
  to_array(a, v);
#pragma unroll
  for (int k = 0; k < E; ++k) top = max_nan(top, fabsf(v[k]));
  return top;
}

// How a launch is laid out: S rows of a unit's ring; bytes of a unit's ring, and of what it has behind it.
struct Plan {
  Phase phase;
  int S, ring_bytes, unit_bytes;
};

// Sum or maximum over a unit; `k`: which of the reductions of a row, `odd`: the row's parity.
template <bool kWarp>
struct Reduce {
  float (*part)[4][32];
  __device__ __forceinline__ float add(float x, int odd, int k) const { return kWarp ? warp_add(x) : cta_add(x, part[odd][k]); }
  __device__ __forceinline__ float max(float x, int odd, int k) const { return kWarp ? lanes_max(x) : cta_max(x, part[odd][k]); }
  // A sum and a maximum together.
  __device__ __forceinline__ void add_max(float& x, float& top, int odd, int k, int l) const {
    x = warp_add(x), top = lanes_max(top);
    if (kWarp) return;
    const unsigned at = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (at == 0) part[odd][k][threadIdx.x >> 5] = x, part[odd][l][threadIdx.x >> 5] = top;
    __syncthreads();
    x = warp_add(at < warps ? part[odd][k][at] : 0.f);
    top = lanes_max(at < warps ? part[odd][l][at] : 0.f);
  }
  __device__ __forceinline__ void sync() const {
    if (kWarp) __syncwarp();
    else __syncthreads();
  }
};

template <bool kWarp, bool kAligned, bool kRing, int E, int C, bool kQuant>
__global__ void __launch_bounds__(kWarp ? 256 : 1024, kWarp ? (C > 8 ? 3 : 4) : 1) rmsnorm_kernel(const p24_rmsnorm_args g, const Plan plan, int* status) {
  __shared__ float part[2][4][32];
  __shared__ Beside<2> beside[kWarp ? 8 : 1];
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int NV = C / E;
  const int lane = threadIdx.x & 31;
  const int per = kWarp ? blockDim.x >> 5 : 1, unit = kWarp ? threadIdx.x >> 5 : 0;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * per + unit, step = static_cast<int64_t>(gridDim.x) * per;
  const bool with_r = g.r != nullptr;
  const Reduce<kWarp> reduce{part};
  Pieces<2, NV, E, kAligned, kRing> row;
  const Split<E, kAligned>& sp = row.sp;
  row.sp.NT = kWarp ? 32 : blockDim.x, row.sp.tid = kWarp ? lane : threadIdx.x, row.sp.d = static_cast<int>(g.d);
  row.in[0] = Matrix(g.x, g.ldx, g.x_dtype);
  row.in[1] = Matrix(g.r, g.ldr, g.r_dtype);
  row.m = with_r ? 2 : 1, row.S = plan.S, row.T = g.T, row.sh = &beside[unit], row.rstd = nullptr, row.status = status;
  // a unit's shared memory: the ring, the weights, its groups' largest magnitudes
  uint8_t* own = smem + unit * plan.unit_bytes;
  row.start(begin, kAligned ? 0 : plan.phase.of(begin), own);
  Weights<NV, E> w;
  float* tops = reinterpret_cast<float*>(own + plan.ring_bytes + (w.kHow == 1 ? sp.NT * C * 4 : 0));
  const int groups = kQuant ? (sp.d + g.group - 1) / g.group : 0;
  const int shift = groups > 1 ? 31 - __clz(g.group) : 30;  // several groups are of a power of two
  const Matrix h_out(g.h, g.ldh, g.r_dtype), y_out(g.y, g.ldy, g.y_dtype);
  const bool hv = sp.fits(h_out, begin), yv = sp.fits(y_out, begin);
  const float inv_d = 1.f / static_cast<float>(sp.d);
  if (kRing) reduce.sync();  // thread 0 has set the ring up
  pdl_wait();
  pdl_trigger();
  if (kRing)
    for (int k = 0; k < plan.S; ++k) row.fill(begin + k * step, k);
  w.start(sp, g.w, g.w_dtype, own + plan.ring_bytes);
  int odd = 0;
  for (int64_t t = begin; t < g.T; t += step, odd ^= 1) {
    Vals<E> h[NV];
    Two sums = both(0.f);
    float e = 0.f;
    if (kRing) row.wait();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      h[i] = filled<E>(0.f);
      if (!sp.has(i)) continue;
      h[i] = row.get(0, i, t);
      if (with_r) {
        const Vals<E> r = row.get(1, i, t);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          h[i].p[k] = h[i].p[k] + r.p[k];
          if (!row.f32(1)) {  // rounded as it is stored
            float x, y;
            apart(h[i].p[k], x, y);
            h[i].p[k] = pair_of(pack_bf16x2(x, y));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < E / 2; ++k) sums = fma(h[i].p[k], h[i].p[k], sums);
    }
    if (sp.has_edge()) {
      e = row.edge(0, t);
      if (with_r) {
        e += row.edge(1, t);
        if (!row.f32(1)) e = rounded_bf16(e);
        put_element(h_out.row(t), row.f32(1), sp.edge, e);
      }
    }
    if (with_r) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sp.has(i)) store_vals<E>(h_out.row(t), row.f32(1), sp.column(i), hv, h[i]);
    }
    float total = fmaf(e, e, sum_of<E>(sums)), top = 0.f;
    if (kQuant && groups == 1) {  // the row's scale with the same meeting of the threads, from the largest |h w|
      top = fabsf(e * w.edge);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!sp.has(i)) continue;
        Vals<E> wi = w.get(sp, i);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) wi.p[k] = wi.p[k] * h[i].p[k];
        top = max_nan(top, top_of(wi));
      }
      reduce.add_max(total, top, odd, 0, 3);
    } else {
      total = reduce.add(total, odd, 0);
    }
    // every thread has read its pieces: the reduction says so
    if (kRing) {
      row.fill(t + plan.S * step, row.stage);
      row.advance();
    }
    float rstd = rsqrtf(total * inv_d + g.eps);
    if (total == __int_as_float(0x7f800000)) {  // squares beyond fp32 (or an infinity): at a scale of 2^-80
      sums = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          const Two small = h[i].p[k] * both(0x1p-80f);
          sums = fma(small, small, sums);
        }
      const float small = e * 0x1p-80f;
      rstd = 0x1p-80f * rsqrtf(reduce.add(fmaf(small, small, sum_of<E>(sums)), odd, 1) * inv_d);
      top = 0.f;
    }
    if (g.rstd && sp.tid == 0) g.rstd[t] = rstd;
    const float by_rstd = kQuant ? -rstd : rstd;  // codes are made from -y
    e = e * by_rstd * w.edge;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!sp.has(i)) continue;
      const Vals<E> wi = w.get(sp, i);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) h[i].p[k] = h[i].p[k] * both(by_rstd) * wi.p[k];
    }
    if (!kQuant) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sp.has(i)) store_vals<E>(y_out.row(t), E == 8 ? 0 : y_out.f32, sp.column(i), yv, h[i]);
      if (sp.has_edge()) put_element(y_out.row(t), E == 8 ? 0 : y_out.f32, sp.edge, e);
      continue;
    }
    uint8_t* y = static_cast<uint8_t*>(g.y) + t * g.ldy;
    const bool qv = kAligned || (reinterpret_cast<uintptr_t>(y + sp.c0) & (E - 1)) == 0;
    float* scales = g.scale + t * g.lds;
    if (groups == 1) {
      if (top >= 0x1p-100f && top <= 0x1p100f) {
        top *= rstd;
      } else {  // h w leaves fp32's range, or is no number
        top = fabsf(e);
#pragma unroll
        for (int i = 0; i < NV; ++i) top = max_nan(top, top_of(h[i]));
        top = reduce.max(top, odd, 2);
      }
      const float sc = scale_of(top);
      const Divisor v = by(sc);
      if (sp.tid == 0) scales[0] = sc;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sp.has(i)) store_e4m3<E>(y, sp.column(i), qv, h[i], v);
      if (sp.has_edge()) y[sp.edge] = e4m3(quotient(e, v));
    } else if (kAligned && g.group <= 32 * E) {
      // a group is some neighbouring lanes' pieces
      const int lanes = g.group / E;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float top = top_of(h[i]);
        for (int k = lanes >> 1; k; k >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, k));
        const float sc = scale_of(top);
        if (!sp.has(i)) continue;
        if ((lane & (lanes - 1)) == 0) scales[sp.column(i) >> shift] = sc;
        store_e4m3<E>(y, sp.column(i), qv, h[i], by(sc));
      }
    } else {
      // A piece meets at most two groups, from column `cut` of it on the second. Magnitudes are ordered as whole
      // numbers, NaN last.
      auto note = [&](int group, float top) { atomicMax(reinterpret_cast<int*>(&tops[group]), __float_as_int(top)); };
      for (int i = sp.tid; i < groups; i += sp.NT) tops[i] = 0.f;
      reduce.sync();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!sp.has(i)) continue;
        const int c = sp.column(i), ga = c >> shift, gb = (c + E - 1) >> shift, cut = ga == gb ? E : (gb << shift) - c;
        float v[E], ta = 0.f, tb = 0.f;
        to_array(h[i], v);
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (k < cut) ta = max_nan(ta, fabsf(v[k]));
          else tb = max_nan(tb, fabsf(v[k]));
        note(ga, ta);
        if (ga != gb) note(gb, tb);
      }
      if (sp.has_edge()) note(sp.edge >> shift, max_nan(fabsf(e), 0.f));
      reduce.sync();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!sp.has(i)) continue;
        const int c = sp.column(i), ga = c >> shift, gb = (c + E - 1) >> shift, cut = ga == gb ? E : (gb << shift) - c;
        store_e4m3<E>(y, c, qv, h[i], by(scale_of(tops[ga])), by(scale_of(tops[gb])), cut);
      }
      if (sp.has_edge()) y[sp.edge] = e4m3(quotient(e, by(scale_of(tops[sp.edge >> shift]))));
      for (int i = sp.tid; i < groups; i += sp.NT) scales[i] = scale_of(tops[i]);
      reduce.sync();  // before the next row's groups
    }
  }
  if (kRing && sp.tid == 0) row.drain(begin < g.T ? (g.T - begin + step - 1) / step : 0);
}

// The gradient. The weight's is summed over a unit's rows in registers (a thread's columns are the same in all
// of them), or where a thread has more than 16 in shared memory, then over a CTA's units, and goes to the CTA's row
// of `parts`.
template <bool kWarp, bool kAligned, bool kRing, int E, int C>
__global__ void __launch_bounds__(kWarp ? 256 : 1024, kWarp ? 3 : 1) rmsnorm_bwd_kernel(const p24_rmsnorm_bwd_args g, const Plan plan, float* parts, int* status) {
  __shared__ float part[2][4][32];
  __shared__ Beside<3> beside[kWarp ? 8 : 1];
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int NV = C / E;
  constexpr bool kHold = C <= 8;   // g and xh stay in registers through the reduction
  constexpr bool kSums = C <= 16;  // and the sums
  const int per = kWarp ? blockDim.x >> 5 : 1, unit = kWarp ? threadIdx.x >> 5 : 0;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * per + unit, step = static_cast<int64_t>(gridDim.x) * per;
  const bool with_r = g.dres != nullptr;
  const Reduce<kWarp> reduce{part};
  Pieces<3, NV, E, kAligned, kRing> row;
  const Split<E, kAligned>& sp = row.sp;
  row.sp.NT = kWarp ? 32 : blockDim.x, row.sp.tid = kWarp ? threadIdx.x & 31 : threadIdx.x, row.sp.d = static_cast<int>(g.d);
  row.in[0] = Matrix(g.h, g.ldh, g.h_dtype);
  row.in[1] = Matrix(g.dy, g.lddy, g.dy_dtype);
  row.in[2] = Matrix(g.dres, g.ldres, g.r_dtype);
  row.m = with_r ? 3 : 2, row.S = plan.S, row.T = g.T, row.sh = &beside[unit], row.rstd = g.rstd, row.status = status;
  // a unit's shared memory: the ring, the weights; the sums take a warp's ring at its end, or are all there is
  uint8_t* own = smem + unit * plan.unit_bytes;
  row.start(begin, kAligned ? 0 : plan.phase.of(begin), own);
  Weights<NV, E> w;
  float* sums = reinterpret_cast<float*>(own);
  const Matrix out(g.dx, g.lddx, g.dx_dtype);
  const bool ov = sp.fits(out, begin);
  const float inv_d = 1.f / static_cast<float>(sp.d);
  Vals<E> acc[kSums ? NV : 1];
  float acc_e = 0.f;
#pragma unroll
  for (int i = 0; i < (kSums ? NV : 1); ++i) acc[i] = filled<E>(0.f);
  if (!kSums && parts)
    for (int c = sp.tid; c < padded(sp.d); c += sp.NT) sums[c] = 0.f;
  if (kRing || !kSums) reduce.sync();  // thread 0 has set the ring up
  pdl_wait();
  pdl_trigger();
  if (kRing)
    for (int k = 0; k < plan.S; ++k) row.fill(begin + k * step, k);
  w.start(sp, g.w, g.w_dtype, own + plan.ring_bytes);
  int odd = 0;
  for (int64_t t = begin; t < g.T; t += step, odd ^= 1) {
    if (kRing) row.wait();
    const float now = kRing ? beside[unit].rstd[row.stage] : g.rstd[t];
    float eh = 0.f, eg = 0.f, er = 0.f;
    if (sp.has_edge()) {
      eh = row.edge(0, t) * now;
      eg = row.edge(1, t);
      if (with_r) er = row.edge(2, t);
      acc_e = fmaf(eg, eh, acc_e);
      eg *= w.edge;
    }
    Vals<E> xh[kHold ? NV : 1], v[kHold ? NV : 1];
    Two dots = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = kHold ? i : 0;
      if (!sp.has(i)) continue;
      xh[u] = row.get(0, i, t);
      v[u] = row.get(1, i, t);
      const Vals<E> wi = w.get(sp, i);
      Vals<E> p;
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        xh[u].p[k] = xh[u].p[k] * both(now);
        if (kSums) acc[kSums ? i : 0].p[k] = fma(v[u].p[k], xh[u].p[k], acc[kSums ? i : 0].p[k]);
        else p.p[k] = v[u].p[k] * xh[u].p[k];
        v[u].p[k] = v[u].p[k] * wi.p[k];
        dots = fma(v[u].p[k], xh[u].p[k], dots);
      }
      if (!kSums && parts) {
        float q[E];
        to_array(p, q);
#pragma unroll
        for (int k = 0; k < E; ++k) sums[padded(sp.column(i) + k)] += q[k];
      }
    }
    const float mean = reduce.add(fmaf(eg, eh, sum_of<E>(dots)), odd, 0) * inv_d;
    if (kRing && !kWarp && plan.S > 2 && t > begin)
      row.fill(t + (plan.S - 1) * step, row.stage == 0 ? plan.S - 1 : row.stage - 1);  // the row before's place
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = kHold ? i : 0;
      if (!sp.has(i)) continue;
      if (!kHold) {
        xh[u] = row.get(0, i, t);
        v[u] = row.get(1, i, t);
        const Vals<E> wi = w.get(sp, i);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) xh[u].p[k] = xh[u].p[k] * both(now), v[u].p[k] = v[u].p[k] * wi.p[k];
      }
      const Vals<E> r = with_r ? row.get(2, i, t) : filled<E>(0.f);
#pragma unroll
      for (int k = 0; k < E / 2; ++k) v[u].p[k] = fma(both(now), fma(xh[u].p[k], both(-mean), v[u].p[k]), r.p[k]);
      store_vals<E>(out.row(t), E == 8 ? 0 : out.f32, sp.column(i), ov, v[u]);
    }
    if (sp.has_edge()) put_element(out.row(t), E == 8 ? 0 : out.f32, sp.edge, fmaf(now, fmaf(eh, -mean, eg), er));
    if (kRing) {
      // A warp's lanes have read the row now, a CTA's threads when they meet in the next row's reduction; with a
      // ring of one or two rows that would be too late (16384 x 8192 fp32, two rows: 347 us, like this 280).
      if (kWarp || plan.S <= 2) {
        reduce.sync();
        row.fill(t + plan.S * step, row.stage);
      }
      row.advance();
    }
  }
  if (kRing && sp.tid == 0) row.drain(begin < g.T ? (g.T - begin + step - 1) / step : 0);
  if (!parts) return;
  float* to = parts + static_cast<int64_t>(blockIdx.x) * sp.d;
  if (kSums && !kWarp) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!sp.has(i)) continue;
      float v[E];
      to_array(acc[kSums ? i : 0], v);
      float* at = to + sp.column(i);
      if (kAligned) {
#pragma unroll
        for (int k = 0; k < E; k += 4) *reinterpret_cast<float4*>(at + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < E; ++k) at[k] = v[k];
      }
    }
    if (sp.has_edge()) to[sp.edge] = acc_e;
    return;
  }
  __syncthreads();  // the rings are done with
  if (kSums) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!sp.has(i)) continue;
      float v[E];
      to_array(acc[kSums ? i : 0], v);
#pragma unroll
      for (int k = 0; k < E; ++k) sums[padded(sp.column(i) + k)] = v[k];
    }
  }
  if (sp.has_edge()) sums[padded(sp.edge)] = acc_e;
  __syncthreads();
  sums = reinterpret_cast<float*>(smem);
  for (int c = threadIdx.x; c < sp.d; c += blockDim.x) {
    float v = sums[padded(c)];
    for (int u = 1; u < per; ++u) v += sums[u * (plan.unit_bytes / 4) + padded(c)];
    to[c] = v;
  }
}

// The gradient of few rows in one launch, for then a second one's 2 us are much of the call: a CTA a row, straight from
// memory, while the first `columns` CTAs add up 64 columns of the weight's gradient each from the inputs, which are read
// twice for that (dx in the place of one of them: those CTAs are a launch of their own). us, and with a ring and parts:
//   16 rows of 128 1.8 and 3.2, of 4096 2.6 and 4.0, of 8192 3.3 and 5.4;  128 rows of 128 3.0 and 3.7, of 4096 3.4 and
//   4.9, of 8192 5.2 and 6.7;  300 rows of 512 5.2 and 4.5, of 2049 5.4 and 8.6, of 4096 5.5 and 6.4, of 8192 9.1 and 8.2
// (With 256 threads 128 rows of 128 took 4.8, with 1024 128 rows of 4096 4.2; with the matrices' types looked at in the
// loop, which kept its loads from going out together, 8.9.)
bool few_rows(int64_t T, int64_t d) { return d <= 8192 && T <= (d > 512 && d <= 4096 ? 2 * sm_count() : 128); }
constexpr unsigned kFewThreads = 512;  // at least
constexpr int kFewColumns = 64;
template <typename Th, typename Td>
__device__ __forceinline__ void few_columns(const p24_rmsnorm_bwd_args& g, int c, int from, int step, float (&s)[2]) {
  const int d = static_cast<int>(g.d), T = static_cast<int>(g.T);
  const Th* h = static_cast<const Th*>(g.h) + c;
  const Td* dy = static_cast<const Td*>(g.dy) + c;
  const bool a = c < d, b = c + 32 < d;
#pragma unroll 8
  for (int t = from; t < T; t += step) {
    const float now = g.rstd[t];
    if (a) s[0] = fmaf(to_float(dy[t * g.lddy]), to_float(h[t * g.ldh]) * now, s[0]);
    if (b) s[1] = fmaf(to_float(dy[t * g.lddy + 32]), to_float(h[t * g.ldh + 32]) * now, s[1]);
  }
}
template <bool kAligned>
__global__ void __launch_bounds__(1024) rmsnorm_bwd_few_kernel(const p24_rmsnorm_bwd_args g, const Phase phase, int columns) {
  __shared__ float part[32];
  __shared__ float sums[kFewColumns][33];
  const int d = static_cast<int>(g.d), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Pieces<3, 2, 4, kAligned, false> row;
  const Split<4, kAligned>& sp = row.sp;
  row.sp.NT = blockDim.x, row.sp.tid = threadIdx.x, row.sp.d = d;
  row.in[0] = Matrix(g.h, g.ldh, g.h_dtype);
  row.in[1] = Matrix(g.dy, g.lddy, g.dy_dtype);
  row.in[2] = Matrix(g.dres, g.ldres, g.r_dtype);
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) < columns) {
    const int c = blockIdx.x * kFewColumns + lane;
    float s[2] = {0.f, 0.f};
    if (row.f32(0)) {
      if (row.f32(1)) few_columns<float, float>(g, c, warp, warps, s);
      else few_columns<float, bf16>(g, c, warp, warps, s);
    } else {
      if (row.f32(1)) few_columns<bf16, float>(g, c, warp, warps, s);
      else few_columns<bf16, bf16>(g, c, warp, warps, s);
    }
    sums[lane][warp] = s[0], sums[lane + 32][warp] = s[1];
    __syncthreads();
    for (int i = warp; i < kFewColumns; i += warps) {
      const float x = warp_add(lane < warps ? sums[i][lane] : 0.f);
      if (lane == 0 && blockIdx.x * kFewColumns + i < d) g.dw[blockIdx.x * kFewColumns + i] = x;
    }
    return;
  }
  const int64_t t = blockIdx.x - columns;
  const bool with_r = g.dres != nullptr;
  row.m = with_r ? 3 : 2;
  row.start(t, kAligned ? 0 : phase.of(t), nullptr);
  const Matrix out(g.dx, g.lddx, g.dx_dtype);
  const bool ov = sp.fits(out, t);
  const float now = g.rstd[t];
  Vals<4> xh[2], v[2], r[2];
  float eh = 0.f, eg = 0.f, er = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r[i] = filled<4>(0.f);
    if (!sp.has(i)) continue;
    xh[i] = row.get(0, i, t), v[i] = row.get(1, i, t);
    if (with_r) r[i] = row.get(2, i, t);
  }
  if (sp.has_edge()) {
    eh = row.edge(0, t), eg = row.edge(1, t);
    if (with_r) er = row.edge(2, t);
  }
  Weights<2, 4> w;
  w.start(sp, g.w, g.w_dtype, nullptr);
  eh *= now, eg *= w.edge;
  Two dots = both(0.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!sp.has(i)) continue;
    const Vals<4> wi = w.get(sp, i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      xh[i].p[k] = xh[i].p[k] * both(now), v[i].p[k] = v[i].p[k] * wi.p[k];
      dots = fma(v[i].p[k], xh[i].p[k], dots);
    }
  }
  const float mean = cta_add(fmaf(eg, eh, sum_of<4>(dots)), part) / static_cast<float>(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!sp.has(i)) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) v[i].p[k] = fma(both(now), fma(xh[i].p[k], both(-mean), v[i].p[k]), r[i].p[k]);
    store_vals<4>(out.row(t), out.f32, sp.column(i), ov, v[i]);
  }
  if (sp.has_edge()) put_element(out.row(t), out.f32, sp.edge, fmaf(now, fmaf(eh, -mean, eg), er));
}

// Column sums of the CTAs' parts [G, d]: 32 columns of a CTA, 32 warps that take
// every 32nd row each. The parts come from L2; 2 to 3 us, most of them the launch and two dependent steps.
__global__ void __launch_bounds__(1024) dweight_kernel(const float* parts, int G, int d, float* dw) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int i = warp; i < G; i += 32) s += parts[static_cast<int64_t>(i) * d + c];
  }
  sh[warp][lane] = s;
  __syncthreads();
  // warp i adds up column i, in one order
  s = warp_add(sh[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = s;
}

// Values of 8-bit codes, bound by memory (16384 x 4096 to bf16 27 us). A CTA: blockDim.x threads with a piece of 8 columns each, blockDim.y rows, U of them for a
// thread. Pieces lie on boundaries of 8 elements, in all rows alike, or row by row: then those at a row's ends are partly
// outside it. Where the two matrices have no common boundaries they are moved element by element.
enum Boundaries { kAlike, kByRow, kNone };
template <typename To, int U, Boundaries kHow>
__global__ void __launch_bounds__(256) dequant8_kernel(const p24_dequant8_args g, const Phase phase, int shift) {
  const int d = static_cast<int>(g.d), piece = blockIdx.y * blockDim.x + threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * U * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  uint2 b[U];
  float sa[U], sb[U];  // a piece meets two groups at most, `cut` columns of it the first
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    const int c = 8 * piece - (kHow == kByRow ? phase.of(t) : 0);
    if (t >= g.T || c >= d) continue;
    const uint8_t* q = static_cast<const uint8_t*>(g.q) + t * g.ldq + c;
    b[u] = make_uint2(0, 0);
    if (kHow != kNone && c >= 0 && c + 8 <= d) {
      b[u] = *reinterpret_cast<const uint2*>(q);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= 0 && c + i < d) (i < 4 ? b[u].x : b[u].y) |= static_cast<uint32_t>(q[i]) << (8 * (i & 3));
    }
    const float* scale = g.scale + t * g.lds;
    sa[u] = scale[max(c, 0) >> shift];
    sb[u] = kHow == kAlike ? sa[u] : scale[min(c + 7, d - 1) >> shift];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t t = t0 + u * blockDim.y;
    const int c = 8 * piece - (kHow == kByRow ? phase.of(t) : 0);
    if (t >= g.T || c >= d) continue;
    const int cut = kHow == kAlike ? 8 : (((max(c, 0) >> shift) + 1) << shift) - c;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h =
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((i < 2 ? b[u].x : b[u].y) >> (16 * (i & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * i] = f.x * (2 * i < cut ? sa[u] : sb[u]);
      v[2 * i + 1] = f.y * (2 * i + 1 < cut ? sa[u] : sb[u]);
    }
    store8(static_cast<To*>(g.y) + t * g.ldy, c, d, kHow != kNone, v);
  }
}

constexpr int kWarpColumns = 512;      // rows of up to so many: a warp each
constexpr size_t kShared = 220 << 10;  // of an SM, for the CTAs' rings

struct Lead {
  const void* p;
  int64_t ld;
  int32_t dtype;
};
// The phases of the first bf16 (or 8-bit) matrix among these, which fp32 ones of the same layout agree with.
Phase phase_of(std::initializer_list<Lead> all) {
  const Lead* lead = all.begin();
  for (const Lead& l : all)
    if (l.p && l.dtype != P24_F32) {
      lead = &l;
      break;
    }
  const uintptr_t at = reinterpret_cast<uintptr_t>(lead->p) / size_of(lead->dtype);
  return Phase{static_cast<int>(at & 7), static_cast<int>(lead->ld & 7)};
}
// Whether the interiors of a matrix begin on 16-byte boundaries (8 bits: of 8) in every row, at the phases of `ph`.
bool in_phase(const Lead& l, int64_t T, Phase ph) {
  const int m = l.dtype == P24_F32 ? 3 : 7;
  return !l.p || (((reinterpret_cast<uintptr_t>(l.p) / size_of(l.dtype) - ph.first) & m) == 0 && (T == 1 || ((l.ld - ph.step) & m) == 0));
}

// What a launch comes to: threads of a CTA, units of it, the plan, shared memory.
struct Shape {
  int NT, per;
  Plan plan;
  size_t smem;
};
// A ring of 2 to 4 rows and as many CTAs as make 1024 threads on an SM, or fewer CTAs, or one row. col_bytes: of a
// column in all matrices that are read; own: what a unit has besides its ring and (16 columns a thread) the weights;
// ahead: how many bytes an SM should have in its rings, 0 for as many as fit. The forward writes as much as it reads
// and is fastest with few (16384 x 8192 bf16, rows of 32 KB: 169 us with 2, 179 with 3, 185 with 4); the gradient
// with all (253, 167, 157).
Shape ring_shape(int d, int C, bool warp, int col_bytes, size_t own, Phase ph, size_t ahead) {
  constexpr int kThreads = 1024;  // of an SM; the registers of a thread allow no more
  Shape z{};
  z.plan.phase = ph;
  z.NT = warp ? 256 : ((d + C - 1) / C + 31) / 32 * 32;
  z.per = warp ? z.NT / 32 : 1;
  const size_t cols = static_cast<size_t>(warp ? 32 : z.NT) * C, row = cols * col_bytes;
  own += C > 8 ? cols * sizeof(float) : 0;
  for (int c = std::max(1, kThreads / z.NT); c >= 1; --c) {
    const size_t room = (kShared / c - 2048) / z.per;  // an SM reserves 1 KB for each CTA, and a CTA has static arrays
    const size_t most = ahead ? std::max<size_t>(2, std::min<size_t>(kMostRows, ahead / (c * z.per * row))) : kMostRows;
    const int S = static_cast<int>(std::min<size_t>(most, room > own ? (room - own) / row : 0));
    if (S < 2 && (c > 1 || S < 1)) continue;
    z.plan.S = S, z.plan.ring_bytes = static_cast<int>(S * row), z.plan.unit_bytes = static_cast<int>(S * row + own);
    z.smem = z.per * static_cast<size_t>(z.plan.unit_bytes);
    break;
  }
  return z;  // S = 0: too wide
}
Shape direct_shape(int d, int C, size_t own, Phase ph) {
  Shape z{};
  z.plan.phase = ph, z.per = 1, z.smem = own;
  z.NT = ((d + C - 1) / C + 31) / 32 * 32;
  return z;
}

// CTAs for T rows: as many as run at once, and units a multiple of 8 so that each has rows of one phase.
template <typename K>
cudaError_t grid_of(K kern, const Shape& z, int64_t T, int64_t most, int64_t* grid) {
  int slots = 0;
  const cudaError_t e = row_kernel_slots(reinterpret_cast<const void*>(kern), z.NT, 1, z.smem, &slots);
  int64_t n = std::min<int64_t>(slots, most);
  if (z.per == 1 && n > 8) n = n / 8 * 8;
  *grid = std::min<int64_t>({(T + z.per - 1) / z.per, n, most});
  return e;
}


// Columns of a thread, 8 or 16. 16 halve the instructions that a row's reduction, its wait and its addresses take
// (164 in all for a warp's 256 columns; issue slots are the forward's bound, 70%), and allow a row of more than 4096
// columns more CTAs on an SM; 8 have twice the ring. us, 8 and 16, rows of bf16 unless said:
//   one matrix to read: 16 (16384 x 4096 51 and 48, x 4095 73 and 46, x 1024 14.0 and 11.8, 8192 x 8192 52 and 43); with
//     fp32 in aligned rows 8 (8192 x 4096 to fp32 35 and 39, x 8192 fp32 86 and 93; x 6290 to fp32 89 and 61)
//   with a residual: 8 (16384 x 4096 81 and 90, x 768 15.3 and 17.6; x 8192 166 and 176), unless they leave the SM a
//     quarter empty (8192 x 5001 70 and 60, beside an fp32 stream 94 and 83)
//   8-bit codes, half as many instructions again: 16 (16384 x 4096 without a residual 78 and 59, with one 91 and 75),
//     with a residual where a row is more than 1024 columns (x 1024 26 and 25, x 768 19.9 and 22.6), or beside an
//     fp32 stream in unaligned rows of more than 4096 (8192 x 6290 135 and 115, x 8192 117 and 134)
//   the gradient: 8 (16384 x 4096 64 and 67, x 1024 22 and 28), 16 without a skip connection's in rows of more than 4096
//     bf16 (8192 x 6290 84 and 70; fp32 125 and 172)
//   few rows: 8, for a row's time is a thread's
int columns_of(int d, int E, bool aligned, bool residual, bool quant, bool gradient, bool few) {
  if (d > 8192) return 16;
  if (few) return 8;
  const int NT = (d + 255) / 256 * 32;
  const bool empty = d > 4096 && 1024 / NT * NT < 768;
  bool more;
  if (gradient) more = E == 8 && d > 4096 && (!residual || empty);
  else if (quant && residual) more = E == 8 ? d > 1024 : !aligned && d > 4096;
  else if (quant) more = E == 8 || d > 1024;
  else more = residual ? empty : E == 8 || !aligned;
  return more ? 16 : 8;
}

template <bool kAligned, int E, bool kQuant>
cudaError_t launch_norm(const p24_rmsnorm_args& g, Phase ph, bool ring, int* status, cudaStream_t s) {
  const int d = static_cast<int>(g.d);
  const int bytes = size_of(g.x_dtype) + (g.r ? size_of(g.r_dtype) : 0);
  const size_t groups = kQuant ? (d + g.group - 1) / g.group : 0, own = (groups * sizeof(float) + 15) / 16 * 16;
  auto go = [&](auto kern, const Shape& z) {
    int64_t grid = 0;
    cudaError_t e = grid_of(kern, z, g.T, INT64_MAX, &grid);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(z.NT), z.smem, s, g, z.plan, status);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (ring && d <= kWarpColumns) {
    if (d <= 256) return go(rmsnorm_kernel<true, kAligned, true, E, 8, kQuant>, ring_shape(d, 8, true, bytes, own, ph, 80 << 10));
    return go(rmsnorm_kernel<true, kAligned, true, E, 16, kQuant>, ring_shape(d, 16, true, bytes, own, ph, 80 << 10));
  }
  const bool few = g.T <= 2 * sm_count();
  const int C = columns_of(d, E, kAligned, g.r != nullptr, kQuant, false, few);
  const Shape z = ring_shape(d, C, false, bytes, own, ph, 80 << 10);
  if (ring && d <= 16384 && z.plan.S > 0)
    return C == 8 ? go(rmsnorm_kernel<false, kAligned, true, E, 8, kQuant>, z) : go(rmsnorm_kernel<false, kAligned, true, E, 16, kQuant>, z);
  return go(rmsnorm_kernel<false, false, false, 4, 32, kQuant>, direct_shape(d, 32, own, ph));
}

// CTAs of the gradient, at most: 8 rows or so of the batch for each, and a multiple of 8 (as units are). Each of them has
// a row of partial sums, and one row of the batch at least.
int64_t bwd_ctas(int64_t T) {
  const int64_t n = std::max<int64_t>(2 * sm_count(), std::min<int64_t>(16 * sm_count(), T / 8));
  return (n + 7) / 8 * 8;
}

template <bool kAligned, int E>
cudaError_t launch_bwd(const p24_rmsnorm_bwd_args& g, Phase ph, bool ring, float* parts, int* status, cudaStream_t s, int64_t* used) {
  const int d = static_cast<int>(g.d);
  const int bytes = size_of(g.h_dtype) + size_of(g.dy_dtype) + (g.dres ? size_of(g.r_dtype) : 0);
  auto go = [&](auto kern, const Shape& z) {
    cudaError_t e = grid_of(kern, z, g.T, bwd_ctas(g.T), used);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(static_cast<unsigned>(*used)), dim3(z.NT), z.smem, s, g, z.plan, parts, status);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  if (ring && d <= kWarpColumns) {
    if (d <= 256) return go(rmsnorm_bwd_kernel<true, kAligned, true, E, 8>, ring_shape(d, 8, true, bytes, 0, ph, 0));
    return go(rmsnorm_bwd_kernel<true, kAligned, true, E, 16>, ring_shape(d, 16, true, bytes, 0, ph, 0));
  }
  const bool few = g.T <= 2 * sm_count();
  const int C = columns_of(d, E, kAligned, g.dres != nullptr, false, true, few);
  const Shape z = ring_shape(d, C, false, bytes, 0, ph, 0);
  if (ring && d <= 16384 && z.plan.S > 0)
    return C == 8 ? go(rmsnorm_bwd_kernel<false, kAligned, true, E, 8>, z) : go(rmsnorm_bwd_kernel<false, kAligned, true, E, 16>, z);
  const size_t sums = ((d + d / 8 + 1) * sizeof(float) + 15) / 16 * 16;
  return go(rmsnorm_bwd_kernel<false, false, false, 4, 32>, direct_shape(d, 32, sums, ph));
}

// Pieces of 8 columns where nothing is fp32; aligned: no edges, and all on their boundaries in every row.
struct Layout {
  bool wide, aligned, ring;
  Phase ph;
};
// in: what the ring reads (the first n); all: with the outputs.
Layout layout_of(std::initializer_list<Lead> all, size_t n, int64_t T, int64_t d, const void* w) {
  Layout l{true, false, true, phase_of(all)};
  for (const Lead& m : all)
    if (m.p && m.dtype == P24_F32) l.wide = false;
  l.aligned = d % 8 == 0 && on16(w) && l.ph.first == 0 && (T == 1 || l.ph.step == 0);
  size_t i = 0;
  for (const Lead& m : all) {
    const bool in = in_phase(m, T, l.ph);
    l.aligned = l.aligned && in;
    if (i++ < n) l.ring = l.ring && in;
  }
  return l;
}

}  // namespace

int64_t rmsnorm_bwd_parts(int64_t T, int64_t d) { return std::min(T, bwd_ctas(T)) * d; }

cudaError_t launch_rmsnorm(const p24_rmsnorm_args& a, int* status, cudaStream_t s) {
  p24_rmsnorm_args g = a;
  if (!g.r) g.r_dtype = g.x_dtype, g.h = nullptr;
  if (g.y_dtype == P24_E4M3 && (g.group == 0 || g.group > g.d)) g.group = static_cast<int32_t>(g.d);
  const Layout l = layout_of({{g.x, g.ldx, g.x_dtype}, {g.r, g.ldr, g.r_dtype}, {g.h, g.ldh, g.r_dtype}, {g.y, g.ldy, g.y_dtype}}, 2, g.T, g.d, g.w);
  auto go = [&](auto quant) {
    constexpr bool kQuant = decltype(quant)::value;
    if (l.wide) return l.aligned ? launch_norm<true, 8, kQuant>(g, l.ph, l.ring, status, s) : launch_norm<false, 8, kQuant>(g, l.ph, l.ring, status, s);
    return l.aligned ? launch_norm<true, 4, kQuant>(g, l.ph, l.ring, status, s) : launch_norm<false, 4, kQuant>(g, l.ph, l.ring, status, s);
  };
  return g.y_dtype == P24_E4M3 ? go(std::true_type()) : go(std::false_type());
}

cudaError_t launch_rmsnorm_bwd(const p24_rmsnorm_bwd_args& g, float* parts, int* status, cudaStream_t s) {
  const Layout l = layout_of({{g.h, g.ldh, g.h_dtype}, {g.dy, g.lddy, g.dy_dtype}, {g.dres, g.ldres, g.r_dtype}, {g.dx, g.lddx, g.dx_dtype}}, 3, g.T, g.d, g.w);
  int64_t used = 0;
  float* to = g.dw ? parts : nullptr;
  cudaError_t e;
  if (few_rows(g.T, g.d)) {
    auto go = [&](unsigned rows, unsigned columns) {
      const dim3 grid(rows + columns), block(std::max(kFewThreads, static_cast<unsigned>((g.d + 255) / 256 * 32)));
      e = l.aligned ? launch_pdl(rmsnorm_bwd_few_kernel<true>, grid, block, 0, s, g, l.ph, static_cast<int>(columns))
                    : launch_pdl(rmsnorm_bwd_few_kernel<false>, grid, block, 0, s, g, l.ph, static_cast<int>(columns));
      if (e == cudaSuccess) count_launch();
      return e;
    };
    const unsigned rows = static_cast<unsigned>(g.T), columns = g.dw ? static_cast<unsigned>((g.d + kFewColumns - 1) / kFewColumns) : 0;
    if (columns == 0 || (g.dx != g.h && g.dx != g.dy)) return go(rows, columns);
    return go(0, columns) != cudaSuccess ? e : go(rows, 0);  // in place: the columns first
  }
  if (l.wide) e = l.aligned ? launch_bwd<true, 8>(g, l.ph, l.ring, to, status, s, &used) : launch_bwd<false, 8>(g, l.ph, l.ring, to, status, s, &used);
  else e = l.aligned ? launch_bwd<true, 4>(g, l.ph, l.ring, to, status, s, &used) : launch_bwd<false, 4>(g, l.ph, l.ring, to, status, s, &used);
  if (e != cudaSuccess || !g.dw) return e;
  const int d = static_cast<int>(g.d);
  e = launch_pdl(dweight_kernel, dim3((d + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(parts), static_cast<int>(used), d, g.dw);
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_dequant8(const p24_dequant8_args& a, cudaStream_t s) {
  p24_dequant8_args g = a;
  if (g.group == 0 || g.group > g.d) g.group = static_cast<int32_t>(g.d);
  const Lead q{g.q, g.ldq, P24_E4M3}, y{g.y, g.ldy, g.y_dtype};
  Phase ph = phase_of({q});
  if (g.T == 1) ph.step = 0;
  const bool phased = in_phase(q, g.T, ph) && in_phase(y, g.T, ph), odd = phased && (ph.first != 0 || ph.step != 0);
  const RowThreads r = row_threads(g.d + (odd ? 7 : 0), 256);
  const dim3 block(r.x, 256 / r.x);
  int shift = 30;  // one group
  if (g.group < g.d)
    for (shift = 5; (1 << shift) < g.group;) ++shift;
  auto go = [&](auto kern, int u) {
    const int64_t rows = static_cast<int64_t>(u) * block.y;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>((g.T + rows - 1) / rows), r.chunks), block, 0, s, g, ph, shift);
    if (e == cudaSuccess) count_launch();
    return e;
  };
  // 4 rows a thread where that leaves 8 CTAs for each SM
  const bool many = g.T * r.x * r.chunks >= 256 * 8 * 4 * sm_count();
  auto how = [&](auto type) {
    using To = decltype(type);
    if (!phased) return go(dequant8_kernel<To, 1, kNone>, 1);
    if (odd) return many ? go(dequant8_kernel<To, 4, kByRow>, 4) : go(dequant8_kernel<To, 1, kByRow>, 1);
    return many ? go(dequant8_kernel<To, 4, kAlike>, 4) : go(dequant8_kernel<To, 1, kAlike>, 1);
  };
  return g.y_dtype == P24_BF16 ? how(bf16()) : how(float());
}

}  // namespace p24
