// logprobs_kernels.cu -- log probabilities of given tokens, entropy and top alternatives of
// rows of logits, and the gradient of the first two.
//
//   x = (z - m) / tau,  m = max z,  s = sum exp(x),  p = exp(x) / s
//   logp = x[token] - ln s        H = ln s - (1/s) sum exp(x) x
//   dz = (1/tau) [ dlogp (delta - p) - dentropy p (ln p + H) ]
//
//  logprobs_kernel      a cluster per row (head_rows.cuh): one pass with a running maximum and
//                       sums per thread, joined over the CTA and the cluster. The alternatives
//                       come from a second look at few vectors: the k-th largest of the threads'
//                       maxima is a lower bound of the k-th largest logit, so only parts whose
//                       maximum reaches it can hold alternatives. Those parts (a thread's share
//                       of one stage or a few) are read again, from L2, the elements that reach
//                       the bound are listed, and each one's place is the number of listed ones
//                       before it. Where the list overflows because many logits tie at the bound,
//                       the ones above it are listed and the rest taken in order of position, if the
//                       bound shows the tied value: any negative one in bf16; in fp32 -inf, and the
//                       lowest finite value in shares of up to kItems parts. Other ties go through
//                       an exact selection, five walks over the share.
//  logprobs_bwd_kernel  elementwise from the saved statistics.
//
// Bound: HBM, one read of the logits (and one write of the gradient). Measured on GB300, of the
// 6.69 TB/s of a plain copy: scores of 4096 x 50257 bf16 64 to 66 us, 0.93 to 0.96; gradient of
// the same rows with entropy 133 us, 0.92, of 1000 x 32003 fp32 42 us, 0.91; entropy and top 64 of
// 8192 x 131072 409 us, 0.79 (the alternatives' searches are a fifth of the instructions, and the
// walk waits for them; top 20 357 us, 0.90); one row of 32000 with 20 alternatives 7.0 us, of which
// 2.4 us are the walk and the rest the alternatives' dependent steps. The search is a fixed cost a
// row, which shorter rows hide less: top 64 of 4096 x 50257 131 us, 0.47, top 20 101 us, 0.61, none 65;
// top 5 of 8192 x 1001 51 us, 0.05, none 16. Exact selections: 16 x 50257 fp32 with 12 live entries
// 36 us masked by -1e9, 11 by -inf; 1000 x 50257 621 and 48 us.
#include <algorithm>
#include <type_traits>

#include "head_rows.cuh"

namespace p24 {
namespace {

// ---------------------------------------------------------------- top k
// Order of the logits as an unsigned key: larger key first; NaN above +inf, -0 equal to +0.
// Every key is above 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
// Key and position in one number that orders both: ties go to the lower position.
__device__ __forceinline__ uint64_t entry(uint32_t key, int i) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int entry_pos(uint64_t e) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e)); }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return static_cast<uint32_t>(e >> 32); }

// With alternatives (20.5 KB for them). Top 64 of 8192 x 131072: 409 us; 427 with 320 or 256 threads
// and 3 CTAs on an SM, 472 with 192 and 5, 465 with 256 and 2. Fewer threads have fewer maxima, so
// more candidates; more threads pay more for each search.
using Long = Layout<256, 4, 4, 2>;
// With alternatives, where an SM has no more than two CTAs: registers to spare. Top 20 of one row of
// 32000 6.9 us, 7.6 in Long; of 256 rows of 50257 with 200 tokens allowed 15.6 us, 19.4.
using Few = Layout<256, 2, 4, 2>;
// Without: scores of 4096 x 50257 64 us; 75 with 256 threads and 4 CTAs, 82 with 512 and 2.
using LongPlain = Layout<192, 5, 4, 3>;
// Gradients: 2048 x 131072 173 us with all of 128 to 512 threads and 16 to 24 KB stages, 191 with 8 KB.
using LongGrad = Layout<192, 4, 8, 2>;
// Rows of up to kShortRow vectors, where there are more than SMs: 8192 x 1001 with 5 alternatives
// 51 us in 128 threads and 6 CTAs, 60 with 8; without 18 us with 8, 20 with 6.
using Short = Layout<128, 6, 2, 4>;
using ShortPlain = Layout<128, 8, 2, 4>;
constexpr int kShortRow = 1024;

constexpr int kList = 1024;  // candidates listed before something else has to be done
constexpr int kParts = 16;   // parts a thread's share of a row has for the second look
constexpr int kItems = 1024; // parts looked at a second time before something else has to be done

template <int NT>
struct TopShared {
  uint64_t list[kList + 32];  // candidates, and zeros after them
  // upper half of the largest element of each thread's parts; rows of 9 words: no bank conflicts
  uint16_t part[NT][kParts + 2];
  uint16_t item[kItems];      // parts to look at: thread * kParts + part
  uint32_t hist[256];
  int warp[16];
  uint32_t low[16], high[16];
  uint32_t prefix;
  int left;                   // how many of the elements equal to the prefix are still to be taken
  int n, items;               // entries listed, parts to look at
};

// Step `i` of a walk over a row part in order of position: step 0 the elements before the
// interior, then tiles of NT interior vectors, last the elements after it. Gives a thread's
// elements of the step (the rest -inf), their number and the first one's position.
template <typename T, int NT>
__device__ __forceinline__ int walk_step(const RowPart<T>& p, int i, int steps, float (&x)[Vec<T>::N], int& pos) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  if (i > 0 && i < steps - 1) {
    const int v = p.lo + (i - 1) * NT + tid;
    if (v >= p.hi) return 0;
    const uint4 r = p.body[v];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = elem_of<T>(r, j);
    pos = p.vec_pos(v);
    return N;
  }
  const int e = i == 0 ? tid : p.head + tid;
  if (e >= (i == 0 ? min(p.head, p.edges) : p.edges)) return 0;
  pos = p.edge_pos(e);
  x[0] = to_f32(p.row[pos]);
  return 1;
}

// The first k elements of a row part that has at least k, unordered, into sh.list[0, k):
// a radix selection of the k-th key, 8 bits a pass, then the elements above it and, in
// order of position, as many equal to it as are needed. All threads; ends with a barrier.
template <typename T, int NT>
__device__ __noinline__ void select_exact(const RowPart<T>& p, int k, TopShared<NT>& sh) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int steps = 2 + (p.hi - p.lo + NT - 1) / NT;
  walk_sync<NT>();
  if (tid == 0) {
    sh.prefix = 0;
    sh.left = k;
    sh.n = 0;
  }
  uint32_t mask = 0;
  for (int shift = 24; shift >= 32 - 8 * static_cast<int>(sizeof(T)); shift -= 8) {
    for (int i = tid; i < 256; i += NT) sh.hist[i] = 0;
    walk_sync<NT>();
    const uint32_t prefix = sh.prefix;
    // a thread adds equal digits up before it touches their counter: rows that come here have many
    uint32_t digit = 0, run = 0;
    for (int i = 0; i < steps; ++i) {
      float x[N];
      int pos;
      const int n = walk_step<T, NT>(p, i, steps, x, pos);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j >= n) continue;
        const uint32_t key = order_key(x[j]), d = (key >> shift) & 255u;
        if ((key & mask) != prefix) continue;
        if (d != digit) {
          if (run) atomicAdd(&sh.hist[digit], run);
          digit = d;
          run = 0;
        }
        ++run;
      }
    }
    if (run) atomicAdd(&sh.hist[digit], run);
    walk_sync<NT>();
    if (warp == 0) {
      // lane l holds the counters of digits 255 - 8 l down to 248 - 8 l
      int own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += static_cast<int>(sh.hist[255 - 8 * lane - i]);
      int before = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, before, d);
        if (lane >= d) before += y;
      }
      before -= own;
      const int left = sh.left;
      __syncwarp();
      if (before < left && left <= before + own) {
        int i = 0, here = left - before;
        for (; static_cast<int>(sh.hist[255 - 8 * lane - i]) < here; ++i) here -= static_cast<int>(sh.hist[255 - 8 * lane - i]);
        sh.left = here;
        sh.prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
      }
    }
    mask |= 255u << shift;
    walk_sync<NT>();
  }
  const uint32_t kth = sh.prefix;
  const int left = sh.left;
  int equal_before = 0;
  for (int i = 0; i < steps; ++i) {
    float x[N];
    int pos = 0;
    const int n = walk_step<T, NT>(p, i, steps, x, pos);
    uint32_t eq = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= n) continue;
      const uint32_t key = order_key(x[j]);
      if ((key & mask) > kth) sh.list[atomicAdd(&sh.n, 1)] = entry(key, pos + j);  // fewer than k of them
      if ((key & mask) == kth) eq |= 1u << j;
    }
    // the place of this thread's equal elements among all of the part's
    const int mine = __popc(eq);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += y;
    }
    if (lane == 31) sh.warp[warp] = incl;
    walk_sync<NT>();
    int before = equal_before + incl - mine;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += sh.warp[w];
      equal_before += sh.warp[w];
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if ((eq >> j) & 1u) {
        if (before < left) sh.list[k - left + before] = entry(order_key(x[j]), pos + j);
        ++before;
      }
    walk_sync<NT>();
  }
}

// Element i of a row part, counted in order of position.
template <typename T>
__device__ __forceinline__ int nth_pos(const RowPart<T>& p, int i) {
  const int head = p.edges > 0 ? p.head : 0, inner = (p.hi - p.lo) * Vec<T>::N;
  return i < head ? i : i - head < inner ? p.vec_pos(p.lo) + i - head : p.tail0 + i - head - inner;
}

// List the elements of this CTA whose key is at least `from`: from the threads' parts that can
// hold any, whose vectors all threads read together. own16: the upper half of the key of the
// thread's largest element. Returns the number found; more than kList if there is no room. All
// threads; sh.n and sh.items are 0 and a barrier lies behind that; ends with a barrier.
template <typename T, typename L>
__device__ __forceinline__ int list_from(const RowPart<T>& p, uint32_t from, uint32_t own16, int stages, int shift,
                                         TopShared<L::NT>& sh) {
  constexpr int N = Vec<T>::N, NT = L::NT;
  static_assert(kParts * NT <= 65536, "an item is 16 bits");
  static_assert(NT >= kTopMax, "k threads' maxima bound the k-th element");
  const int tid = threadIdx.x;
  const float least = from ? key_value(from) : ninf();  // as numbers: no NaN comes here
  auto list = [&](float x, int pos) {
    const int at = atomicAdd(&sh.n, 1);
    if (at < kList) sh.list[at] = entry(order_key(x), pos);
  };
  if (own16 >= (from >> 16) && own16 > 0) {
    // a part's upper half stands for a number no smaller than the bound's where an element is (a
    // negative one's lower half only takes it further down)
    const float bound = least > 0.f ? __uint_as_float(__float_as_uint(least) & 0xffff0000u) : least;
    const uint32_t* parts = reinterpret_cast<const uint32_t*>(sh.part[tid]);
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < kParts / 2; ++i) {
      const uint32_t w = parts[i];
      if (__uint_as_float(w << 16) >= bound) found |= 1u << (2 * i);
      if (__uint_as_float(w & 0xffff0000u) >= bound) found |= 2u << (2 * i);
    }
    found &= (2u << ((stages - 1) >> shift)) - 1u;
    for (; found; found &= found - 1) {
      const int at = atomicAdd(&sh.items, 1);
      if (at < kItems) sh.item[at] = static_cast<uint16_t>(tid * kParts + __ffs(found) - 1);
    }
    if (tid < p.edges) {
      const int pos = p.edge_pos(tid);
      const float x = to_f32(p.row[pos]);
      if (x >= least) list(x, pos);
    }
  }
  walk_sync<NT>();
  const int items = sh.items;
  if (items > kItems) return kList + 1;
  const int lg = shift + 31 - __clz(L::SV);  // log2 of a part's vectors
  for (int i = tid; i < items << lg; i += NT) {
    const int item = sh.item[i >> lg];
    const int v = p.lo + ((item % kParts << lg) + (i & ((1 << lg) - 1))) * NT + item / kParts;
    if (v >= p.hi) continue;
    const uint4 r = p.body[v];
    uint32_t found = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (elem_of<T>(r, j) >= least) found |= 1u << j;
    for (; found; found &= found - 1) {
      const int j = __ffs(found) - 1;
      const uint32_t w = j < N / 2 ? (j < N / 4 ? r.x : r.y) : (j < 3 * N / 4 ? r.z : r.w);
      list(sizeof(T) == 4 ? __uint_as_float(w) : __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16), p.vec_pos(v) + j);
    }
  }
  walk_sync<NT>();
  return sh.n;
}

// This CTA's first min(k, its elements) elements, unordered, into sh.list; returns how many are
// listed there (at least those). own16: the upper half of the order key of the thread's largest
// element (0: it has none); odd: the row holds a NaN or +inf, which the maxima do not show. All
// threads; ends with a barrier.
template <typename T, typename L>
__device__ __forceinline__ int top_of_part(const RowPart<T>& p, int k, uint32_t own16, bool odd, int stages, int shift,
                                           TopShared<L::NT>& sh) {
  constexpr int NT = L::NT;
  const int tid = threadIdx.x, lane = tid & 31;
  const int have = (p.hi - p.lo) * Vec<T>::N + p.edges;
  if (k > have) k = have;
  if (k == 0) return 0;
  if (odd) {
    select_exact<T, NT>(p, k, sh);
    return k;
  }
  // the largest bound that k threads' maxima reach; 0 where fewer than k threads have elements
  const uint32_t low = __reduce_min_sync(~0u, own16), high = __reduce_max_sync(~0u, own16);
  if (lane == 0) sh.low[tid >> 5] = low, sh.high[tid >> 5] = high;
  if (tid == 0) sh.n = sh.items = 0;
  walk_sync<NT>();
  uint32_t lo = __reduce_min_sync(~0u, sh.low[lane % (NT / 32)]), hi = __reduce_max_sync(~0u, sh.high[lane % (NT / 32)]);
  while (lo < hi) {
    const uint32_t mid = (lo + hi + 1) / 2;
    if (walk_count<NT>(own16 >= mid) >= k) lo = mid;
    else hi = mid - 1;
  }
  int n = 0;
  const bool masked = lo == 0x7fu || lo == 0x80u;  // a bound of -inf or of the lowest finite values
  if (!masked) {
    n = list_from<T, L>(p, lo << 16, own16, stages, shift, sh);
    if (n <= kList) return n;
  }
  // Many ties at the bound: in bf16 the bound is one value; in fp32 two masking values are looked
  // for, -inf and the lowest finite one. List what is above, then take ties from the front.
  const uint32_t tie = sizeof(T) == 2 ? ((lo & 0x8000u) ? lo << 16 : lo << 16 | 0xffffu) : lo == 0x7fu ? 0x7fffffu : lo << 16;
  if (sizeof(T) == 2 || masked) {
    walk_sync<NT>();
    if (tid == 0) sh.n = sh.items = 0;
    walk_sync<NT>();
    n = list_from<T, L>(p, tie + 1, own16, stages, shift, sh);
    if (n >= k && n <= kList) return n;
    walk_sync<NT>();
    // Ties complete a list that holds everything above them. One that ran out of room does not (and
    // sh.n is no count of what is above them then: an fp32 bound of 0x80 covers values next to the
    // lowest one, whose parts alone can be too many).
    if (n < k) {
      if (tid < 32) {
        constexpr int kEach = 4, kSteps = 32;
        for (int step = 0; step < kSteps && n < k; ++step) {
          const int i0 = step * 32 * kEach + lane;
          float x[kEach];
#pragma unroll
          for (int j = 0; j < kEach; ++j) x[j] = i0 + 32 * j < have ? to_f32(p.row[nth_pos(p, i0 + 32 * j)]) : 0.f;
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const uint32_t same = __ballot_sync(~0u, i0 + 32 * j < have && order_key(x[j]) == tie);
            const int at = n + __popc(same & ((1u << lane) - 1));
            if (((same >> lane) & 1u) && at < k) sh.list[at] = entry(tie, nth_pos(p, i0 + 32 * j));
            n += __popc(same);
          }
        }
        if (lane == 0) sh.n = min(n, k);
      }
      walk_sync<NT>();
      n = sh.n;
      if (n == k) return n;
    }
  }
  select_exact<T, NT>(p, k, sh);
  return k;
}

// kTop: with alternatives.
template <typename T, bool kEntropy, bool kTop, typename L>
__global__ void __launch_bounds__(L::kThreads, L::kCtas) logprobs_kernel(const p24_logprobs_args g, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT;
  extern __shared__ __align__(128) uint4 ring_data[];
  __shared__ RingShared<L::S> ring_sh;
  __shared__ JoinShared joins;
  TopShared<NT>& top = *reinterpret_cast<TopShared<NT>*>(reinterpret_cast<char*>(ring_data) + L::kRing);  // kTop
  // kTop and more ranks than one: the ranks' lists in rank 0, [row parity][rank][k], in order
  uint64_t* best = reinterpret_cast<uint64_t*>(&top + 1);
  __shared__ uint64_t best_in[2];
  const int tid = threadIdx.x, V = static_cast<int>(g.V), k = static_cast<int>(g.k);
  const int ranks = cluster_ranks(), rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const float tau = g.temperature, c = kLog2e / tau;
  const T* logits = static_cast<const T*>(g.logits);
  const int stages = row_stages(V / Vec<T>::N, ranks, L::kStage);
  int shift = 0;  // stages to a part of the second look, a power of two
  while (kTop && (stages - 1) >> shift >= kParts) ++shift;
  R ring{logits, g.ldz, blockIdx.x / ranks, gridDim.x / ranks, g.T, V, rank, ranks, stages, 1, ring_data, &ring_sh, status};
  if (tid == 0) {
    join_init(joins, ranks);
    for (int i = 0; i < 2; ++i) mbar_init(&best_in[i], ranks);
  }
  ring.start();
  begin(ranks);
  if (tid >= NT) {
    if (tid == NT) ring.run();
    return;
  }

  float edge = load_edge(RowPart<T>(logits + ring.first * g.ldz, V, rank, ranks));
  int64_t r = 0;
  for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
    const RowPart<T> p(logits + t * g.ldz, V, rank, ranks);
    float z_tok = 0.f;
    bool has_tok = false;
    if (g.logp && tid == 0 && rank == 0) {
      const int tok = g.tokens[t];
      has_tok = tok >= 0 && tok < V;
      if (has_tok) z_tok = to_f32(p.row[tok]);
    }
    Walk<kEntropy> w;
    float part_max = ninf();
    if (tid < p.edges) w.add_one(edge, c);
    if (t + ring.step < g.T) edge = load_edge(RowPart<T>(logits + (t + ring.step) * g.ldz, V, rank, ranks));
    for (int at = 0; at < stages; ++at) {
      const uint4* data = ring.wait();
      const int n = p.hi - p.lo - at * L::kStage;
      uint32_t mr = Vec<T>::kFill;
      R::each(data, n, [&](const uint4& x, int) { mr = max_vec<T>(mr, x); });
      const float vm = max_of<T>(mr);
      w.raise(vm, c);
      if constexpr (kTop) {
        part_max = fmaxf(part_max, vm);
        if (((at + 1) & ((1 << shift) - 1)) == 0 || at + 1 == stages) {
          top.part[tid][at >> shift] = static_cast<uint16_t>(__float_as_uint(part_max) >> 16);
          part_max = ninf();
        }
      }
      const F2 a = w.a;
      R::each(data, n, [&](const uint4& x, int) { w.template add<T>(x, c); });
      if (kEntropy && w.lost()) {
        w.a = a;
        R::each(data, n, [&](const uint4& x, int) { w.template add_floored<T>(x, c); });
      }
      ring.release();
    }
    const float own_max = w.m;
    const bool own = p.lo + tid < p.hi || tid < p.edges;
    Sums u = w.sums(), unused{0.f, 0.f, 0.f};
    row_join<kEntropy, false, NT>(u, c, unused, c, joins, r, rank, ranks, &ring_sh.abort, status);
    const float ls = u.s == 0.f ? ninf() : logf(u.s);
    // ln of the probability of a logit; a row with nothing above -inf has none
    auto logp = [&](float z) { return u.s == 0.f ? ninf() : (z - u.m) / tau - ls; };
    if (tid == 0 && rank == 0) {
      if (g.stats) {
        g.stats[2 * t] = u.m;
        g.stats[2 * t + 1] = ls;
      }
      if (g.logp) g.logp[t] = has_tok ? logp(z_tok) : 0.f;
      if (kEntropy) g.entropy[t] = u.s == 0.f ? 0.f : ls - u.a / (u.s * tau);
    }
    if constexpr (kTop) {
      auto put = [&](uint64_t e, int place) {
        g.top_idx[t * k + place] = entry_pos(e);
        g.top_logp[t * k + place] = logp(key_value(entry_key(e)));
      };
      int n = top_of_part<T, L>(p, k, own ? order_key(own_max) >> 16 : 0u, !(u.s == u.s), stages, shift, top);
      // Each entry's place is the number of entries before it. Of several ranks, each sends its first
      // k to rank 0, which does the same with those: one copy of the code for both.
      const bool sends = *const_cast<volatile int*>(&ring_sh.abort) == 0;
#pragma unroll 1
      for (int last = ranks > 1 ? 0 : 1; last < 2; ++last) {
        if (tid < 32) top.list[n + tid] = 0;  // no entry is before any other there: a multiple of 32
        walk_sync<NT>();
        const int all = !last ? max(n, k) : n, sub = tid & 3;
#pragma unroll 1
        for (int i0 = 0; i0 + (tid >> 5) * 8 < all; i0 += NT / 4) {  // four lanes to an entry
          const int i = i0 + (tid >> 2);
          const uint64_t e = i < n ? top.list[i] : 0;
          int place = 0;
#pragma unroll 1
          for (int j0 = sub; j0 < n; j0 += 32) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) place += top.list[j0 + j] > e;
          }
          place += __shfl_xor_sync(~0u, place, 1);
          place += __shfl_xor_sync(~0u, place, 2);
          if (i >= n) place = i;  // what a share lacks of k entries comes after all others
          if (sub != 0 || place >= k || i >= all) continue;
          if (last) put(e, place);
          else if (sends) store_remote(remote(best + ((r & 1) * ranks + rank) * kTopMax + place, 0), e);
        }
        walk_sync<NT>();  // the list and the parts' maxima are free
        if (last) break;
        if (tid == 0) {
          if (sends) arrive_remote(&best_in[r & 1], 0);
          top.n = 0;
        }
        if (rank != 0) break;
        wait_cluster(&best_in[r & 1], (r >> 1) & 1, &ring_sh.abort, status);
        walk_sync<NT>();
        // each list's first k / ranks (rounded up) are k entries or more: what is below all of them is out
        const uint64_t* lists = best + (r & 1) * ranks * kTopMax;
        uint64_t least = ~uint64_t(0);
        const int first = ((k + ranks - 1) >> (31 - __clz(ranks))) - 1;
#pragma unroll 1
        for (int i = 0; i < ranks; ++i) least = min(least, lists[i * kTopMax + first]);
#pragma unroll 1
        for (int i = tid; i < ranks * kTopMax; i += NT) {
          const uint64_t e = i % kTopMax < k ? lists[i] : 0;
          if (e != 0 && e >= least) top.list[atomicAdd(&top.n, 1)] = e;
        }
        walk_sync<NT>();
        n = top.n;
      }
      for (int i = V + tid; rank == 0 && i < k; i += NT) {  // fewer entries than alternatives asked for
        g.top_idx[t * k + i] = -1;
        g.top_logp[t * k + i] = ninf();
      }
    }
  }
  end(ranks, &ring_sh.abort);
}

// The gradient, elementwise: a CTA takes parts of rows.
template <typename T, bool kEntropy, typename L>
__global__ void __launch_bounds__(L::kThreads, L::kCtas) logprobs_bwd_kernel(const p24_logprobs_args g, int parts, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT;
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 ring_data[];
  __shared__ RingShared<L::S> ring_sh;
  const int tid = threadIdx.x, V = static_cast<int>(g.V), part = blockIdx.x % parts;
  const float tau = g.temperature, c1 = 1.f / tau;
  const T* logits = static_cast<const T*>(g.logits);
  struct Row {
    int tok;
    float m, ls, dl, dh, H, edge;
  };
  const int stages = row_stages(V / N, parts, L::kStage);
  R ring{logits, g.ldz, blockIdx.x / parts, gridDim.x / parts, g.T, V, part, parts, stages, 1, ring_data, &ring_sh, status};
  ring.start();
  begin(1);
  if (tid >= NT) {
    if (tid == NT) ring.run();
    return;
  }
  auto row_of = [&](int64_t t) {
    Row r;
    r.tok = g.tokens ? g.tokens[t] : -1;
    if (r.tok >= V) r.tok = -1;
    r.m = g.stats[2 * t];
    r.ls = g.stats[2 * t + 1];
    r.dl = g.dlogp ? g.dlogp[t] : 0.f;
    r.dh = kEntropy ? g.dentropy[t] : 0.f;
    r.H = kEntropy ? g.entropy[t] : 0.f;
    r.edge = load_edge(RowPart<T>(logits + t * g.ldz, V, part, parts));
    return r;
  };
  Row row = row_of(ring.first);
  for (int64_t t = ring.first; t < g.T; t += ring.step) {
    const RowPart<T> p(logits + t * g.ldz, V, part, parts);
    const Row now = row;
    if (t + ring.step < g.T) row = row_of(t + ring.step);
    T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(p.row) & 15u);
    const bool none = now.ls == ninf();  // a row with nothing above -inf
    const float m = none ? 0.f : now.m, ls = none ? 0.f : now.ls;
    const float dl = (!none && now.tok >= 0) ? now.dl * c1 : 0.f;
    const float dh = (kEntropy && !none) ? now.dh * c1 : 0.f;
    const float k0 = kEntropy ? -(dl + dh * now.H) : -dl;  // dz = p (k0 - dh ln p) + dl delta
    const F2 m2 = f2(-m, -m), c2 = f2(c1, c1), ls2 = f2(-ls, -ls), e2 = f2(kLog2e, kLog2e);
    auto grad = [&](F2 z) {
      F2 lp = fma2(add2(z, m2), c2, ls2);
      if constexpr (kEntropy) {
        float a, b;
        split(lp, a, b);
        lp = f2(floored(a), floored(b));
      }
      const F2 q = ex2x2(mul2(lp, e2));
      return mul2(q, kEntropy ? fma2(f2(-dh, -dh), lp, f2(k0, k0)) : f2(k0, k0));
    };
    if (tid < p.edges) {
      const int pos = p.edge_pos(tid);
      float y, unused;
      split(grad(f2(now.edge, now.edge)), y, unused);
      out[pos] = static_cast<T>(y + (pos == now.tok ? dl : 0.f));
    }
    for (int at = 0; at < stages; ++at) {
      const uint4* data = ring.wait();
      const int n = p.hi - p.lo - at * L::kStage;
      R::each(data, n, [&](const uint4& x, int u) {
        F2 y[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) y[j] = grad(pair<T>(x, j));
        const int i0 = p.vec_pos(p.lo + at * L::kStage + u * NT + tid);
        if (now.tok >= i0 && now.tok < i0 + N) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j)
            y[j] = add2(y[j], f2(now.tok == i0 + 2 * j ? dl : 0.f, now.tok == i0 + 2 * j + 1 ? dl : 0.f));
        }
        store_vec(out, i0, aligned, pack_vec<T>(y));
      });
      ring.release();
    }
  }
}

// As row_split, with alternatives. A share costs its vectors (0.63 us for 1000) in each round. Several
// of them cost a second join, about 2200 vectors; each CTA that an SM has costs about 2300 more, for
// the searches of an SM's CTAs hold each other up. Of several shares 3 fit on an SM at a time, of whole
// rows 4. Measured with 1, 2, 4, 8 shares: 32 rows of 131072 16.2, 12.4, 9.9, 10.5 us; 64 of 32000 8.1,
// 8.2, 9.1, 16.8; 200 of 131072 20.5, 19.2 with the first two.
int top_split(int64_t T, int64_t vecs) {
  const int64_t sms = sm_count();
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMaxRanks && (n == 1 || vecs >= n * int64_t(128)); n *= 2) {
    const int64_t rounds = (T * n + (n > 1 ? 3 : 4) * sms - 1) / ((n > 1 ? 3 : 4) * sms);
    const int64_t cost = rounds * (vecs / n) + (n > 1 ? 2200 : 0) + (T * n + sms - 1) / sms * 2300;
    if (cost < least) least = cost, best = n;
  }
  return best;
}

template <typename T, bool kEntropy, bool kTop>
cudaError_t launch_logprobs_as(const p24_logprobs_args& g, int* status, cudaStream_t s) {
  using L = std::conditional_t<kTop, Long, LongPlain>;
  const int64_t vecs = g.V / Vec<T>::N;
  auto smem = [&](auto layout, int ranks) {
    using M = decltype(layout);
    return M::kRing + (kTop ? sizeof(TopShared<M::NT>) + (ranks > 1 ? 2 * ranks * kTopMax * sizeof(uint64_t) : 0) : 0);
  };
  if (vecs <= kShortRow && g.T > sm_count()) {
    using M = std::conditional_t<kTop, Short, ShortPlain>;
    return launch_rows(logprobs_kernel<T, kEntropy, kTop, M>, M::kThreads, g.T, 1, smem(M(), 1), s, g, status);
  }
  // Without alternatives, 1000 vectors a CTA: 16 x 32000 2.9 us over 8 CTAs a row, 4.1 whole; 256 x 131072
  // 11.6 over 2, 13.9 whole, 15.4 over 4; 450 x 32000 6.2 whole, 8.8 over 2.
  const int ranks = kTop ? top_split(g.T, vecs) : row_split(g.T, vecs, sm_count() * L::kCtas, kMaxRanks, 1000);
  if (kTop && g.T * ranks <= sm_count() * Few::kCtas)
    return launch_rows(logprobs_kernel<T, kEntropy, kTop, std::conditional_t<kTop, Few, L>>, Few::kThreads, g.T, ranks,
                       smem(Few(), ranks), s, g, status);
  return launch_rows(logprobs_kernel<T, kEntropy, kTop, L>, L::kThreads, g.T, ranks, smem(L(), ranks), s, g, status);
}

template <typename T, bool kEntropy>
cudaError_t launch_logprobs_bwd_as(const p24_logprobs_args& g, int* status, cudaStream_t s) {
  const int64_t vecs = g.V / Vec<T>::N;
  if (vecs <= kShortRow)
    return launch_parts(logprobs_bwd_kernel<T, kEntropy, ShortPlain>, ShortPlain::kThreads, g.T, 1, ShortPlain::kRing, s, g, 1,
                        status);
  // A CTA costs an SM about 256 vectors where L2 holds logits and gradient (450 rows of 32000 bf16 7.7 us;
  // 8.7 at 64, in fours), less where memory is the bound (1000 of 32003 fp32 42 us in fours; 44 whole).
  const int64_t fixed = g.T * vecs * 32 > (int64_t(128) << 20) ? 64 : 256;
  const int parts = row_split(g.T, vecs, sm_count() * LongGrad::kCtas, 64, fixed);
  return launch_parts(logprobs_bwd_kernel<T, kEntropy, LongGrad>, LongGrad::kThreads, g.T, parts, LongGrad::kRing, s, g, parts,
                      status);
}

template <typename T>
cudaError_t launch_logprobs_type(const p24_logprobs_args& g, int* st, cudaStream_t s) {
  if (g.k > 0) return g.entropy ? launch_logprobs_as<T, true, true>(g, st, s) : launch_logprobs_as<T, false, true>(g, st, s);
  return g.entropy ? launch_logprobs_as<T, true, false>(g, st, s) : launch_logprobs_as<T, false, false>(g, st, s);
}

}  // namespace

cudaError_t launch_logprobs(const p24_logprobs_args& g, int* status, cudaStream_t s) {
  return g.dtype == P24_BF16 ? launch_logprobs_type<__nv_bfloat16>(g, status, s) : launch_logprobs_type<float>(g, status, s);
}

cudaError_t launch_logprobs_bwd(const p24_logprobs_args& g, int* status, cudaStream_t s) {
  if (g.dtype == P24_BF16)
    return g.dentropy ? launch_logprobs_bwd_as<__nv_bfloat16, true>(g, status, s)
                      : launch_logprobs_bwd_as<__nv_bfloat16, false>(g, status, s);
  return g.dentropy ? launch_logprobs_bwd_as<float, true>(g, status, s) : launch_logprobs_bwd_as<float, false>(g, status, s);
}

}  // namespace p24
