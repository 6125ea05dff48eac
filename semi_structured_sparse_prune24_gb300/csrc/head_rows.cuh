// head_rows.cuh -- what the language-model head's row kernels share: how a row of logits is
// split over threads and CTAs, its softmax sums, and how they are joined.
//
// A row of V elements at any element alignment is its interior, nint aligned 16-byte vectors
// of N elements starting `head` elements in, and at most 2 (N - 1) edge elements before and
// after it. A cluster of C CTAs takes a row together: rank r the interior vectors
// from r ceil(nint / C) on, rank 0 the edges too (one per thread).
//
// A CTA's share of its rows comes through a ring of stages in shared memory, filled by bulk
// copies (cp.async.bulk) that run ahead of the threads by the ring's length, over row ends too:
// loads are under way while the CTA reduces, waits and stores. A warp of its own issues the
// copies. Measured against that (the loss of 4096 rows of 50257, 112 us then): with the last warp
// to read a stage refilling it the slowest warp of every stage issued the next copy as well, and
// each stage took about 0.9 us longer; loads into registers, refilled as they were used, gave
// 2.3 ms against 0.75 ms for the loss and gradient of 8192 x 131072.
//
// Several CTAs of 2 to 8 warps share an SM, each at another point of another row: a row's
// reductions and waits (about 2 us) hide behind the others' walks. One CTA of 16 or 24 warps on an
// SM took 1.2 to 1.9 ms for that gradient.
#pragma once
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "p24_internal.h"
#include "p24_ptx.cuh"

namespace p24 {
namespace {

// How a kernel is laid out on an SM: kCtas CTAs of NT threads that walk the rows and a warp that
// fills their ring, of S stages of SV vectors per thread.
template <int NT_, int kCtas_, int SV_, int S_>
struct Layout {
  static constexpr int NT = NT_, kCtas = kCtas_, SV = SV_, S = S_, kWarps = NT_ / 32;
  static constexpr int kThreads = NT + 32;
  static constexpr int kStage = NT * SV;          // vectors of a stage
  static constexpr int kRing = S * kStage * 16;   // bytes
};

constexpr int kTopMax = P24_TOPK_MAX;
constexpr int kMaxRanks = 8;                  // the portable cluster size
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(x, -1e30) that keeps a NaN: a difference of -inf (a masked logit) becomes finite, so
// that its product with exp = 0 is 0 and not NaN.
__device__ __forceinline__ float floored(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fF149F2CA;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction: a gradient's vector of 8 bf16 takes 37 instructions
// instead of 50 (of them 8 exponentials, at a quarter of the issue rate).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(F2 p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p.v));
}
__device__ __forceinline__ F2 add2(F2 p, F2 q) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(p.v), "l"(q.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 p, F2 q) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(p.v), "l"(q.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 p, F2 q, F2 s) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(p.v), "l"(q.v), "l"(s.v));
  return r;
}
__device__ __forceinline__ F2 ex2x2(F2 p) {
  float x, y;
  split(p, x, y);
  return f2(ex2(x), ex2(y));
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }

// ---------------------------------------------------------------- vectors of 16 bytes
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  static constexpr uint32_t kFill = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
};

// Element pairs j of a vector as fp32: j < N / 2.
template <typename T>
__device__ __forceinline__ F2 pair(const uint4& r, int j) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return j == 0 ? f2(__uint_as_float(r.x), __uint_as_float(r.y)) : f2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
}

template <typename T>
__device__ __forceinline__ float elem_of(const uint4& r, int j) {
  float x, y;
  split(pair<T>(r, j >> 1), x, y);
  return (j & 1) ? y : x;
}

// The larger elements of two registers of a vector, NaN dropped; and the largest element of one.
template <typename T>
__device__ __forceinline__ uint32_t max_raw(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 2) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  } else {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
}
// Of a vector and what was found before.
template <typename T>
__device__ __forceinline__ uint32_t max_vec(uint32_t a, const uint4& r) {
  return max_raw<T>(max_raw<T>(a, max_raw<T>(r.x, r.y)), max_raw<T>(r.z, r.w));
}
template <typename T>
__device__ __forceinline__ float max_of(uint32_t a) {
  if constexpr (sizeof(T) == 2)
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  else
    return fmaxf(__uint_as_float(a), ninf());  // a NaN is dropped here too
}

// ---------------------------------------------------------------- a row's parts
template <typename T>
struct RowPart {
  const T* row;
  const uint4* body;  // the interior's first vector
  int head, tail0;    // the interior covers elements [head, tail0)
  int lo, hi;         // this CTA's interior vectors
  int edges;          // this CTA's edge elements (rank 0: all of the row's)

  // ranks: a power of two
  __device__ __forceinline__ RowPart(const T* r, int V, int rank, int ranks) {
    constexpr int N = Vec<T>::N;
    const int a = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    head = min(a ? N - a : 0, V);
    const int nint = (V - head) / N;
    tail0 = head + nint * N;
    row = r;
    body = reinterpret_cast<const uint4*>(r + head);
    const int each = (nint + ranks - 1) >> (31 - __clz(ranks));
    lo = min(nint, rank * each);
    hi = min(nint, lo + each);
    edges = rank == 0 ? head + V - tail0 : 0;
  }
  __device__ __forceinline__ int edge_pos(int e) const { return e < head ? e : tail0 + e - head; }
  __device__ __forceinline__ int vec_pos(int v) const { return head + v * Vec<T>::N; }
  // whether element i of the row is this CTA's
  __device__ __forceinline__ bool owns(int i) const {
    if (i < head || i >= tail0) return edges > 0;
    const int v = (i - head) / Vec<T>::N;
    return v >= lo && v < hi;
  }
};

template <typename T>
__device__ __forceinline__ float load_edge(const RowPart<T>& p) {
  const int e = static_cast<int>(threadIdx.x);
  return e < p.edges ? to_f32(p.row[p.edge_pos(e)]) : ninf();
}

// ---------------------------------------------------------------- softmax sums
// Sums over part of a row relative to its maximum m: s = sum exp((z - m)/tau) and
// a = sum exp((z - m)/tau) (z - m). s == 0: nothing above -inf yet. c = log2(e) / tau below. The
// difference z - m is formed first: z c - m c would lose it for logits of large magnitude, and
// give NaN for rows whose every logit is the type's lowest value. Everything is fp32; the
// exponential is the hardware's, 2^-22 relative.
struct Sums {
  float m, s, a;
};

// The factor that takes sums at m to the reference `to` >= m; d becomes m - to.
__device__ __forceinline__ float rebase_factor(float m, float to, float c, float& d) {
  d = floored(m - to);
  return ex2(d * c);
}

// A thread's sums while it walks its vectors; two halves that are added at the end.
template <bool kEntropy>
struct Walk {
  float m;
  F2 s, a;

  __device__ __forceinline__ Walk() : m(ninf()), s(f2(0.f, 0.f)), a(f2(0.f, 0.f)) {}

  __device__ __forceinline__ void raise(float vm, float c) {  // the running maximum becomes at least vm
    if (vm > m) {
      if (m > ninf()) {
        float d;
        const float r = rebase_factor(m, vm, c, d);
        if constexpr (kEntropy) a = mul2(fma2(s, f2(d, d), a), f2(r, r));
        s = mul2(s, f2(r, r));
      }
      m = vm;
    }
  }
  __device__ __forceinline__ float ref() const { return m > ninf() ? m : 0.f; }

  // The elements of a vector, of which none is above m.
  template <typename T>
  __device__ __forceinline__ void add(const uint4& r, float c) {
    const float ref_ = -ref();
    const F2 off = f2(ref_, ref_), c2 = f2(c, c);
#pragma unroll
    for (int j = 0; j < Vec<T>::N / 2; ++j) {
      const F2 t = add2(pair<T>(r, j), off);
      const F2 e = ex2x2(mul2(t, c2));
      s = add2(s, e);
      if constexpr (kEntropy) a = fma2(e, t, a);
    }
  }
  // Whether an element of -inf (0 times -inf), or a NaN, has gone into `a`: then `a` of the vectors
  // since it was last right is summed again with the difference floored. Looked at once a stage:
  // at each vector it took 6 of its 48 instructions.
  __device__ __forceinline__ bool lost() const {
    float x, y;
    split(a, x, y);
    return x + y != x + y;
  }
  template <typename T>
  __device__ __forceinline__ void add_floored(const uint4& r, float c) {
    const float ref_ = -ref();
    const F2 off = f2(ref_, ref_), c2 = f2(c, c);
#pragma unroll
    for (int j = 0; j < Vec<T>::N / 2; ++j) {
      float x, y;
      split(add2(pair<T>(r, j), off), x, y);
      const F2 t = f2(floored(x), floored(y));
      a = fma2(ex2x2(mul2(t, c2)), t, a);
    }
  }
  __device__ __forceinline__ void add_one(float x, float c) {
    raise(x, c);
    const float t = floored(x - ref());
    const float e = ex2(t * c);
    s = add2(s, f2(e, 0.f));
    if constexpr (kEntropy) a = add2(a, f2(e * t, 0.f));
  }
  __device__ __forceinline__ Sums sums() const {
    Sums u{m, 0.f, 0.f};
    float x, y;
    split(s, x, y);
    u.s = x + y;
    split(a, x, y);
    u.a = x + y;
    return u;
  }
};

// The larger of two maxima ignores a NaN, as the running maximum does.
__device__ __forceinline__ float warp_max(float m) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// The sums of kParts parts, one per lane (and again from lane kParts on), in every lane. The
// order of the additions is fixed.
template <bool kEntropy, int kParts = 32>
__device__ __forceinline__ Sums warp_join(Sums u, float c) {
  const float m = warp_max(u.m);
  float d, r = rebase_factor(u.m, m, c, d);
  if (u.s == 0.f) r = 0.f, d = 0.f;
  float a = (u.a + u.s * d) * r, s = u.s * r;
#pragma unroll
  for (int i = kParts / 2; i; i >>= 1) {
    s += __shfl_xor_sync(~0u, s, i);
    if constexpr (kEntropy) a += __shfl_xor_sync(~0u, a, i);
  }
  return Sums{m, s, a};
}

__device__ __forceinline__ Sums join(Sums u, Sums v, float c) {
  const float m = fmaxf(u.m, v.m);
  float d;
  const float ru = rebase_factor(u.m, m, c, d), rv = rebase_factor(v.m, m, c, d);
  return Sums{m, (u.s == 0.f ? 0.f : u.s * ru) + (v.s == 0.f ? 0.f : v.s * rv), 0.f};
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ int cluster_ranks() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return static_cast<int>(n);
}
// The address of `p` (shared memory of this CTA) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_remote(uint32_t a, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t a, uint64_t x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}

// Arrive at the barrier `bar` of CTA `rank` of the cluster.
__device__ __forceinline__ void arrive_remote(const uint64_t* bar, int rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote(bar, rank)) : "memory");
}

// Whole-cluster barrier that threads of a warp may reach apart.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

struct JoinShared {
  Sums warp[2][2][16];         // by row parity and sum: the warps'
  Sums rank[2][2][kMaxRanks];  // and the cluster's CTAs'
  uint64_t arrived[2];         // a row's CTAs have written theirs
};

// One thread, before the CTA's (or the cluster's) first barrier.
__device__ __forceinline__ void join_init(JoinShared& sh, int ranks) {
  for (int i = 0; i < 2; ++i) mbar_init(&sh.arrived[i], ranks);
}

// Bounded wait for a phase that threads of other CTAs of the cluster complete.
__device__ __forceinline__ void wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return;
    if (i == 0) t0 = global_ns();
    if ((i & 255u) == 255u) {
      if (*abort) return;
      if (global_ns() - t0 > P24_WAIT_NS) {
        *abort = 1;
        p24_record_timeout(status, bar);
        return;
      }
    }
  }
}

// Barrier of the NT threads of a CTA that walk its rows; and how many of them `on` holds for.
template <int NT>
__device__ __forceinline__ void walk_sync() {
  named_bar_sync(1, NT);
}
template <int NT>
__device__ __forceinline__ int walk_count(bool on) {
  int n;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "bar.red.popc.u32 %0, 1, %2, p;\n\t}"
      : "=r"(n)
      : "r"(static_cast<int>(on)), "r"(NT)
      : "memory");
  return n;
}

// The sums of row r of a CTA, in each of the NT threads that walk it, and
// over all CTAs of its cluster. kTwo: of two kinds at once. Buffers and barriers take turns from
// row to row: a CTA writes to one of them again only when every CTA is past the row between.
template <bool kEntropy, bool kTwo, int NT>
__device__ __forceinline__ void row_join(Sums& u, float c, Sums& v, float cv, JoinShared& sh, int64_t r, int rank, int ranks,
                                         volatile int* abort, int* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, par = r & 1;
  u = warp_join<kEntropy>(u, c);
  if (kTwo) v = warp_join<false>(v, cv);
  if (lane == 0) {
    sh.warp[par][0][warp] = u;
    if (kTwo) sh.warp[par][1][warp] = v;
  }
  walk_sync<NT>();
  // NT / 32 parts, or the next power of two with empty ones
  constexpr int kWarps = NT / 32, kParts = kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : 16;
  const Sums none{ninf(), 0.f, 0.f};
  const int from = lane % kParts;
  u = warp_join<kEntropy, kParts>(from < kWarps ? sh.warp[par][0][from] : none, c);
  if (kTwo) v = warp_join<false, kParts>(from < kWarps ? sh.warp[par][1][from] : none, cv);
  if (ranks > 1) {
    if (warp == 0 && lane < ranks && *abort == 0) {
      const uint32_t to = remote(&sh.rank[par][0][rank], lane);
      store_remote(to, u.m);
      store_remote(to + 4, u.s);
      if constexpr (kEntropy) store_remote(to + 8, u.a);
      if (kTwo) {
        const uint32_t to1 = remote(&sh.rank[par][1][rank], lane);
        store_remote(to1, v.m);
        store_remote(to1 + 4, v.s);
      }
      arrive_remote(&sh.arrived[par], lane);
    }
    wait_cluster(&sh.arrived[par], (r >> 1) & 1, abort, status);
    const int i = lane % kMaxRanks;
    u = warp_join<kEntropy, kMaxRanks>(i < ranks ? sh.rank[par][0][i] : none, c);
    if (kTwo) v = warp_join<false, kMaxRanks>(i < ranks ? sh.rank[par][1][i] : none, cv);
  }
}

// ---------------------------------------------------------------- the ring
template <int S>
struct RingShared {
  uint64_t full[S];    // a stage's data has arrived
  uint64_t empty[S];   // every warp has read it
  int abort;           // a wait ran out (the device status word says so)
};

// The stages a CTA walks: for each of its rows (row r of it is row first + r step), `visits`
// times the `stages` parts of L::kStage vectors of its share. Stage q of that sequence sits in
// slot q % S. A warp of its own fills the slots (one lane issues the copies), so that the others
// only wait for data and say when they have read it.
template <typename T, typename L>
struct Ring {
  static constexpr int S = L::S, kStage = L::kStage, kWalkers = L::NT;
  const T* logits;
  int64_t ld, first, step, rows;
  int V, rank, ranks, stages, visits;
  uint4* data;
  RingShared<S>* sh;
  int* status;
  // the next stage: of the reading warps to read, of the filling one to fill
  int slot = 0;
  uint32_t parity = 0;
  // the filling lane's: what is left of the current row's share, the visit of it, the row
  const uint4* from = nullptr;
  int left = 0, at = 0, visit = 0;
  int64_t row = 0, fills = 0;

  // All threads of the CTA; ends with a barrier, and no global memory is touched before.
  __device__ __forceinline__ void start() {
    if (threadIdx.x == 0) {
      sh->abort = 0;
      for (int i = 0; i < S; ++i) {
        mbar_init(&sh->full[i], 1);
        mbar_init(&sh->empty[i], L::kWarps);
      }
      fence_barrier_init();
      fence_proxy_async_smem();
    }
    __syncthreads();
  }

  // ---- the reading warps
  // The next stage's data, once it is there: vector u of this thread is at u * L::NT.
  __device__ __forceinline__ uint4* wait() {
    p24_wait(&sh->full[slot], parity, &sh->abort, status);
    return data + slot * kStage + threadIdx.x;
  }
  // f(vector, u) for this thread's vectors of a stage that holds n (or, past the ring's stage
  // size, all of them).
  template <typename F>
  __device__ __forceinline__ static void each(const uint4* at, int n, F&& f) {
    if (n >= kStage) {
#pragma unroll
      for (int u = 0; u < L::SV; ++u) f(at[u * L::NT], u);
    } else {
#pragma unroll 1
      for (int u = 0; u * L::NT + static_cast<int>(threadIdx.x) < n; ++u) f(at[u * L::NT], u);
    }
  }
  // This warp has read the current stage: on to the next.
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->empty[slot]);
    advance();
  }
  __device__ __forceinline__ void advance() {
    if (++slot == S) {
      slot = 0;
      parity ^= 1;
    }
  }

  // ---- the filling lane
  __device__ __forceinline__ bool more() const { return first + row * step < rows; }
  __device__ __forceinline__ void fill() {
    if (at == 0) {
      const RowPart<T> p(logits + (first + row * step) * ld, V, rank, ranks);
      from = p.body + p.lo;
      left = p.hi - p.lo;
    }
    const int n = min(left, kStage);
    if (n <= 0) {  // rows of one matrix can differ by a vector: nothing to copy for this one
      mbar_arrive(&sh->full[slot]);
    } else {
      mbar_arrive_expect_tx(&sh->full[slot], n * 16u);
      // what is read for the last time need not stay in L2, what comes again should
      uint64_t policy;
      if (visit + 1 < visits)
        asm("createpolicy.fractional.L2::evict_last.b64 %0;" : "=l"(policy));
      else
        asm("createpolicy.fractional.L2::evict_first.b64 %0;" : "=l"(policy));
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
              smem_u32(data + slot * kStage)),
          "l"(from), "r"(n * 16u), "r"(smem_u32(&sh->full[slot])), "l"(policy)
          : "memory");
    }
    ++fills;
    advance();
    from += kStage;
    left -= kStage;
    if (++at == stages) {
      at = 0;
      if (++visit == visits) {
        visit = 0;
        ++row;
      }
    }
  }
  // Fill everything, each slot once it has been read. The slots are free to begin with.
  __device__ __forceinline__ void run() {
    while (more()) {
      if (fills >= S && !p24_wait(&sh->empty[slot], parity ^ 1, &sh->abort, status)) break;
      fill();
    }
    finish();
  }
  // After an expired wait, copies may still be on their way into this CTA's shared memory.
  __device__ __forceinline__ void finish() const {
    if (*reinterpret_cast<volatile int*>(&sh->abort) == 0) return;
    for (int64_t i = fills > S ? fills - S : 0; i < fills; ++i) p24_wait_quiet(&sh->full[i % S], (i / S) & 1);
  }
};

// Elements w exp((z - m)/tau - l) (+ w1 exp(z - m - l1)): a gradient's terms in p, with off =
// -l log2(e) and off1 = -l1 log2(e).
struct Terms {
  float m, c, off, w, off1, w1;

  template <bool kTwo>
  __device__ __forceinline__ float one(float z) const {
    const float d = z - m;
    float y = w * ex2(fmaf(d, c, off));
    if constexpr (kTwo) y = fmaf(w1, ex2(fmaf(d, kLog2e, off1)), y);
    return y;
  }
  template <bool kTwo>
  __device__ __forceinline__ F2 two(F2 z) const {
    const F2 d = add2(z, f2(-m, -m));
    F2 y = mul2(f2(w, w), ex2x2(fma2(d, f2(c, c), f2(off, off))));
    if constexpr (kTwo) y = fma2(f2(w1, w1), ex2x2(fma2(d, f2(kLog2e, kLog2e), f2(off1, off1))), y);
    return y;
  }
};

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const F2 (&y)[Vec<T>::N / 2]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < Vec<T>::N / 2; ++j) {
    float a, b;
    split(y[j], a, b);
    if constexpr (sizeof(T) == 2) {
      w[j] = pack_bf16x2(a, b);
    } else {
      w[2 * j] = __float_as_uint(a);
      w[2 * j + 1] = __float_as_uint(b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Store a vector at element i0 of an output row; `aligned`: the row has the logits' alignment.
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int i0, bool aligned, const uint4& r) {
  if (aligned) {
    *reinterpret_cast<uint4*>(row + i0) = r;
  } else {
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) row[i0 + j] = static_cast<T>(elem_of<T>(r, j));
  }
}

// What every kernel here begins with, in all threads, once its shared memory is set up: the
// cluster's CTAs run before one of them writes to another's shared memory, and the stream's
// previous kernel has finished before global memory is touched.
__device__ __forceinline__ void begin(int ranks) {
  if (ranks > 1) cluster_barrier();
  pdl_wait();
  pdl_trigger();
}

// And ends with, in whole warps. A CTA that no wait ran out in has had all that the others of its
// cluster ever send it. One that gave up sends nothing more, and stays for what may still come
// until all others have ended or given up as well. (A barrier in every call took 0.6 us of 12: 48
// rows of 131072 fp32, top 8.)
__device__ __forceinline__ void end(int ranks, volatile int* abort) {
  if (__any_sync(~0u, ranks > 1 && *abort != 0)) cluster_barrier();
}

// ---------------------------------------------------------------- launch
// `blocks` CTAs in clusters of `ranks`, with programmatic stream serialization: a call's set-up
// overlaps the end of the kernel before it, which is a good part of a call on few rows.
template <typename... KArgs, typename... Args>
cudaError_t launch_blocks(void (*kern)(KArgs...), int64_t blocks, int threads, int ranks, size_t smem, cudaStream_t s,
                          Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) count_launch();
  return e;
}

// The shared memory that spreads `n` clusters of `ranks` CTAs evenly, where `slots` of them would
// fit: so much that no SM takes more CTAs than its share. Left alone, the CTAs pile up on the SMs
// that are free first, with the stream's previous kernel still on the others: loss and gradient of 256
// rows of 32000 8.4 us instead of 10.1, scores of 256 x 131072 13.8 instead of 16.5, of 200 x 32000 5.2
// instead of 6.8. One CTA for each SM stays as it is: another kernel's CTAs fit beside it.
inline size_t even_smem(const void* kern, int threads, int ranks, int64_t n, int64_t slots, size_t smem) {
  constexpr size_t kPerSm = 228 << 10, kReserved = 1024, kStatic = 8 << 10;  // a CTA's own, and room for its static part
  const size_t share = (n * ranks + sm_count() - 1) / sm_count();
  if (share < 2 || n == slots) return smem;
  const size_t more = kPerSm / (share + 1);  // and the reserved part: share + 1 CTAs do not fit
  if (smem >= more || more + kReserved + kStatic > kPerSm / share) return smem;
  int fit = 0;
  const cudaError_t e = row_kernel_slots(kern, threads, ranks, more, &fit);
  return e == cudaSuccess && fit >= n ? more : smem;
}

// A persistent grid of clusters of `ranks` CTAs over `rows` items.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), int threads, int64_t rows, int ranks, size_t smem, cudaStream_t s,
                        Args&&... args) {
  int slots = 0;
  const cudaError_t e = row_kernel_slots(reinterpret_cast<const void*>(kern), threads, ranks, smem, &slots);
  if (e != cudaSuccess) return e;
  const int64_t n = std::min<int64_t>(rows, slots);
  smem = even_smem(reinterpret_cast<const void*>(kern), threads, ranks, n, slots, smem);
  return launch_blocks(kern, n * ranks, threads, ranks, smem, s, std::forward<Args>(args)...);
}

// Over how many CTAs (a power of two up to `most`) to split rows of `vecs` vectors, T of them on
// `slots` CTAs at a time: the rows of the last round leave CTAs idle, and each CTA that an SM has
// costs as much as `fixed` vectors.
inline int row_split(int64_t T, int64_t vecs, int64_t slots, int most, int64_t fixed) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= most && (n == 1 || vecs >= n * int64_t(128)); n *= 2) {
    const int64_t cost = (T * n + slots - 1) / slots * (vecs / n) + (T * n + sm_count() - 1) / sm_count() * fixed;
    if (cost < least) least = cost, best = n;
  }
  return best;
}
// As launch_rows, over T rows in `parts` parts: CTA b takes part b % parts of rows.
template <typename... KArgs, typename... Args>
cudaError_t launch_parts(void (*kern)(KArgs...), int threads, int64_t T, int parts, size_t smem, cudaStream_t s, Args&&... args) {
  int slots = 0;
  const cudaError_t e = row_kernel_slots(reinterpret_cast<const void*>(kern), threads, 1, smem, &slots);
  if (e != cudaSuccess) return e;
  const int64_t n = std::min<int64_t>(T, std::max(1, slots / parts)) * parts;
  smem = even_smem(reinterpret_cast<const void*>(kern), threads, 1, n, slots, smem);
  return launch_blocks(kern, n, threads, 1, smem, s, std::forward<Args>(args)...);
}

// Stages that the longest share of a row of `vecs` vectors takes.
__host__ __device__ constexpr int row_stages(int64_t vecs, int ranks, int per_stage) {
  const int64_t n = (vecs + ranks - 1) / ranks;
  return n > per_stage ? static_cast<int>((n + per_stage - 1) / per_stage) : 1;
}

}  // namespace
}  // namespace p24
