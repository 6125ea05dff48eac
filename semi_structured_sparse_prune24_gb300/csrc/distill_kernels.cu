// distill_kernels.cu -- distillation of rows of student logits from a teacher's top-K list,
// with the label's cross entropy: loss, gradient, or both in one pass.
//
//   p = softmax(z / tau), q = the teacher's probabilities of the listed columns
//   kl = sum_list q (ln q - ln p) [+ q_r (ln q_r - ln p_r): the rest of the vocabulary as one bucket]
//   tau dkl/dz = Q p - q on the list, p (Q - q_r / p_r) off it, Q = sum q + q_r
//   ce = ln s1 - (z_label - m), dce/dz = softmax(z) - delta
//
//  distill_kernel      a cluster per row (head_rows.cuh). With the bucket the listed elements
//                      stay out of the pass's sums (p_r by subtraction would lose all digits
//                      when the list holds nearly everything). The gradient follows from the
//                      row's second way through the ring (from L2); the listed columns and the
//                      label are then stored again with their own terms.
//  distill_bwd_kernel  the gradient alone, elementwise from the saved statistics. Where p_r is
//                      below e^-64 (all of the bucket masked by a finite value, say) they have
//                      too few digits of it, and the row's sum off the list is taken again.
//
// Bound: HBM, one read of the logits (and one write of the gradient). Measured on GB300, of the
// 6.69 TB/s of a plain copy: loss and gradient of 8192 x 131072 bf16 with 64 entries and the bucket
// 748 us, 0.86 (the rest: rows in flight that L2 loses before their second visit, and the clusters'
// joins); of 1023 x 50257 fp32 at two temperatures 82 us, 0.75 (rows come out uneven on 456
// CTAs); loss alone of 4096 x 50257 67 us, 0.91; gradient alone of 2048 x 131072 173 us, 0.93.
#include <algorithm>
#include <type_traits>

#include "head_rows.cuh"
#include "p24_chain.h"

namespace p24 {
namespace {

// ---------------------------------------------------------------- the teacher's list
// One row's list and arguments in shared memory. Two of them take turns: a warp of its own fills
// one, a row ahead, while the others work on the row of the other.
struct ListShared {
  int idx[kTopMax];   // column, -1 for an absent entry
  float z[kTopMax];   // the student's logit there
  float q[kTopMax];   // the teacher's probability
  float q_sum, q_rest;
  float top, s_list;  // the listed logits' maximum and their sum of exp((z - top) / tau)
  int label;          // -1: none
  int label_listed;
  float z_label, dkl, dce;
};

constexpr int kPerLane = kTopMax / 32;

// A warp's copy of a list, entry j in lane j % 32, slot j / 32.
struct ListRegs {
  int idx[kPerLane];
  float val[kPerLane];

  __device__ __forceinline__ void load(const p24_distill_args& g, int64_t t) {
    const int K = static_cast<int>(g.K), lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int j = lane + 32 * i;
      idx[i] = -1;
      val[i] = ninf();
      if (j < K) {
        idx[i] = g.top_idx[t * K + j];
        val[i] = g.top_val[t * K + j];
      }
    }
  }
};

// Row t's list with the teacher's probabilities, and its arguments, into shared memory: one warp.
// own: of the logits only those of this CTA's share are wanted.
template <typename T>
__device__ __forceinline__ void list_row(const p24_distill_args& g, int64_t t, const RowPart<T>& p, bool own, ListShared& sh,
                                         ListRegs& r) {
  const int K = static_cast<int>(g.K), V = static_cast<int>(g.V), lane = threadIdx.x & 31;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  const float tau = g.temperature;
  r.load(g, t);
  int label = g.labels ? g.labels[t] : -1;
  if (label >= V || label < 0) label = -1;
  // what an in-place gradient overwrites is read here, before
  const float z_label = label >= 0 && (!own || p.owns(label)) ? to_f32(p.row[label]) : 0.f;
  const float dkl = g.dkl ? g.dkl[t] : 0.f, dce = g.dce && label >= 0 ? g.dce[t] : 0.f;
  float z[kPerLane], q[kPerLane];
  float vtop = ninf(), ztop = ninf();
  bool listed = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const bool on = r.idx[i] >= 0 && r.idx[i] < V;
    z[i] = on && (!own || p.owns(r.idx[i])) ? to_f32(p.row[r.idx[i]]) : ninf();
    q[i] = on ? r.val[i] : ninf();
    vtop = fmaxf(vtop, q[i]);
    listed |= on && r.idx[i] == label;
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) ztop = fmaxf(ztop, z[i]);
  vtop = warp_max(vtop);
  ztop = warp_max(ztop);
  float sum = 0.f, s = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const float x = q[i];
    // absent: 0; a NaN stays one; the list's softmax at the temperature, or the probabilities as they are
    q[i] = x != x ? x : x == ninf() ? 0.f : expf(tail ? x : (x - vtop) / tau);
    sum += q[i];
    if (ztop > ninf() || z[i] != z[i]) s += ex2(floored(z[i] - ztop) * (kLog2e / tau));
  }
  sum = warp_sum(sum);
  s = warp_sum(s);
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int j = lane + 32 * i;
    if (j < K) {
      sh.idx[j] = r.idx[i] >= 0 && r.idx[i] < V ? r.idx[i] : -1;
      sh.z[j] = z[i];
      sh.q[j] = !tail && sum != 0.f ? q[i] / sum : q[i];
    }
  }
  listed = __any_sync(~0u, listed);
  if (lane == 0) {
    sh.q_rest = tail ? fmaxf(1.f - sum, 0.f) : 0.f;
    sh.q_sum = tail ? sum : sum != 0.f ? 1.f : 0.f;
    sh.top = ztop;
    sh.s_list = s;
    sh.label = label;
    sh.label_listed = listed;
    sh.z_label = z_label;
    sh.dkl = dkl;
    sh.dce = dce;
  }
}

struct RowStats {
  float m, ls, lr, l1;  // maximum; ln of the sums over all, off the list, over all at temperature 1
  // The sum off the list once more, as a reference and its ln there. Where everything off the list
  // lies far below the maximum (masked by -1e9, say), lr has no digits left for it.
  float rest_m, rest_ls;
};

// A row's gradient: its terms off the list and on it, the factor on q and the label's.
struct RowGrad {
  Terms off, on;
  float wq, wl;
};
__device__ __forceinline__ RowGrad row_grad(const ListShared& sh, bool two, float tau, const RowStats& st) {
  RowGrad r;
  float m = st.m, ls = st.ls, l1 = st.l1, dkl = sh.dkl, dce = sh.dce;
  // a row with nothing above -inf: all terms 0
  const bool none = ls == ninf();
  if (none) m = ls = l1 = dkl = dce = 0.f;
  const float q_rest = st.rest_ls == ninf() ? 0.f : sh.q_rest;  // a bucket in which the student can have nothing is dropped
  r.wq = dkl / tau;
  r.wl = dce;
  r.on.m = m, r.on.c = kLog2e / tau, r.on.off = -ls * kLog2e, r.on.off1 = -l1 * kLog2e;
  r.on.w = r.wq * (sh.q_sum + q_rest);
  r.on.w1 = dce;
  r.off = r.on;
  if (q_rest > 0.f) {
    // Q p - q_r p / p_r = (Q p_r - q_r) times the softmax of what is off the list by itself: neither
    // p nor p_r has to be representable
    const float p_rest = expf(st.lr - ls);
    r.off.m = st.rest_m;
    r.off.off = -st.rest_ls * kLog2e;
    r.off.off1 = ((st.rest_m - m) - l1) * kLog2e;
    r.off.w = r.wq * ((sh.q_sum + q_rest) * p_rest - q_rest);
    if (!two) r.off.w += dce * p_rest;
  } else if (!two) {
    r.off.w += dce;  // one temperature: the label's softmax is p
  }
  if (!two) r.on.w += dce;
  return r;
}

// The gradient's terms off the list, over the next stages of the ring: those of a row.
template <typename T, bool kTwo, typename R>
__device__ __forceinline__ void store_row(R& ring, T* out, bool aligned, const RowPart<T>& p, int stages,
                                          const Terms& terms) {
  constexpr int N = Vec<T>::N, NT = R::kWalkers;
  for (int at = 0; at < stages; ++at) {
    const uint4* data = ring.wait();
    const int v0 = p.lo + at * R::kStage + static_cast<int>(threadIdx.x);
    R::each(data, p.hi - p.lo - at * R::kStage, [&](const uint4& x, int u) {
      F2 y[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) y[j] = terms.template two<kTwo>(pair<T>(x, j));
      store_vec(out, p.vec_pos(v0 + u * NT), aligned, pack_vec<T>(y));
    });
    ring.release();
  }
}

// The listed columns and the label, stored after the rest of the row (and a barrier).
template <typename T, bool kTwo, int NT>
__device__ __forceinline__ void store_listed(T* out, const RowPart<T>& p, const ListShared& sh, int K, const RowGrad& rg) {
  const int label = sh.label;
  for (int j = threadIdx.x; j <= K; j += NT) {
    const int i = j < K ? sh.idx[j] : (sh.label_listed ? -1 : label);
    if (i < 0 || !p.owns(i)) continue;
    float y = j < K ? rg.on.template one<kTwo>(sh.z[j]) - rg.wq * sh.q[j] : rg.off.template one<kTwo>(sh.z_label);
    if (i == label) y -= rg.wl;
    out[i] = static_cast<T>(y);
  }
}

// Loss of 4096 x 50257: 67 us; 76 with 192 threads and 16 KB stages, 69 with 24 KB, 90 with 3 CTAs
// on an SM.
using Loss = Layout<128, 6, 8, 2>;
// Loss and gradient of 8192 x 131072: 750 us; 771 with twice the stages of 16 KB, 757 with 24 KB, 765
// with 192 threads.
using Step = Layout<256, 3, 8, 2>;
using Grad = Layout<192, 4, 8, 2>;
// Rows of up to kShortRow vectors: loss of 8192 x 1001 25 us, 36 with 128 threads and 6 CTAs.
using Short = Layout<64, 10, 4, 2>;
// Gradient of 8192 x 1001 with the bucket 18.6 us; 20.8 with 10 CTAs, whose 63 registers let no more in.
using ShortGrad = Layout<64, 12, 4, 2>;
constexpr int kShortRow = 1024;

// The listed elements of a CTA's share, chained up by the stage and the warp that reads them:
// head[stage * kWarps + warp] is the first entry of the list there (-1: none).
struct Marks {
  int next[kTopMax];
  int lane[kTopMax];   // the reading lane
  int byte[kTopMax];   // and the element's place in the stage, in bytes
  uint32_t edges;      // listed edge elements
};

// Chain up a row's list: one warp. All heads are -1 before.
template <typename T, typename L>
__device__ __forceinline__ void mark_listed(const RowPart<T>& p, const ListRegs& r, int V, Marks& marks, int* head) {
  constexpr int N = Vec<T>::N;
  if ((threadIdx.x & 31) == 0) marks.edges = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int at = r.idx[i], j = (threadIdx.x & 31) + 32 * i;
    if (at < 0 || at >= V || !p.owns(at)) continue;
    if (at >= p.head && at < p.tail0) {
      const int v = (at - p.head) / N - p.lo, in = v % L::kStage, thread = in % L::NT;
      marks.lane[j] = thread & 31;
      marks.byte[j] = in * 16 + (at - p.head) % N * static_cast<int>(sizeof(T));
      marks.next[j] = atomicExch(&head[v / L::kStage * L::kWarps + (thread >> 5)], j);
    } else {
      atomicOr(&marks.edges, 1u << (at < p.head ? at : p.head + at - p.tail0));
    }
  }
}

// What passes between the warp that prepares the lists and the ones that walk the rows, by row
// parity.
struct Handover {
  uint64_t ready[2];  // the list of a row is there
  uint64_t stats[2];  // the row's statistics are there
  uint64_t freed[2];  // the walking warps are done with the list
  RowStats row[2];
};

// kl and ce of row t: one warp.
__device__ __forceinline__ void store_loss(const p24_distill_args& g, int64_t t, const ListShared& sh, const RowStats& st) {
  const int lane = threadIdx.x & 31, K = static_cast<int>(g.K);
  const bool none = st.ls == ninf();  // nothing above -inf
  float kl = 0.f;
  for (int j = lane; j < K; j += 32) {
    const float q = sh.q[j];
    const float lp = none ? ninf() : (sh.z[j] - st.m) / g.temperature - st.ls;
    if (q != 0.f) kl += q * (logf(q) - lp);
  }
  kl = warp_sum(kl);
  if (lane != 0) return;
  const float qr = st.rest_ls == ninf() ? 0.f : sh.q_rest;
  // the factor on the distance first: the distance over tau may be beyond fp32
  if (qr > 0.f) kl += qr * (logf(qr) - (st.rest_ls - st.ls)) + qr / g.temperature * (st.m - st.rest_m);
  g.kl[t] = kl;
  if (g.ce) g.ce[t] = sh.label < 0 ? 0.f : none ? -ninf() : st.l1 - (sh.z_label - st.m);
  if (g.stats) {
    g.stats[4 * t] = st.m;
    g.stats[4 * t + 1] = st.ls;
    g.stats[4 * t + 2] = st.lr;
    g.stats[4 * t + 3] = st.l1;
  }
}

// kGrad: with the gradient. kTwo: the label's softmax (temperature 1) differs from the list's.
// The CTA's last warp prepares the lists and stores the losses, the one before it fills the ring,
// the others walk the rows.
template <typename T, bool kTwo, bool kGrad, typename L>
__global__ void __launch_bounds__(L::kThreads + 32, L::kCtas) distill_kernel(const p24_distill_args g, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT, N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 ring_data[];
  __shared__ RingShared<L::S> ring_sh;
  __shared__ JoinShared joins;
  __shared__ ListShared lists[2];
  __shared__ Marks marks[2];
  __shared__ Handover hand;
  const int tid = threadIdx.x, warp = tid >> 5, V = static_cast<int>(g.V), K = static_cast<int>(g.K);
  const int ranks = cluster_ranks(), rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  const float tau = g.temperature, c = kLog2e / tau;
  const T* logits = static_cast<const T*>(g.logits);
  const int stages = row_stages(V / N, ranks, L::kStage);
  int* heads = reinterpret_cast<int*>(reinterpret_cast<char*>(ring_data) + L::kRing);  // tail: of the marks' chains
  R ring{logits, g.ldz, blockIdx.x / ranks, gridDim.x / ranks, g.T, V, rank, ranks, stages, kGrad ? 2 : 1,
         ring_data, &ring_sh, status};
  if (tid == 0) {
    join_init(joins, ranks);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hand.ready[i], 1);
      mbar_init(&hand.stats[i], 1);
      mbar_init(&hand.freed[i], L::kWarps);
    }
  }
  if (tail)
    for (int i = tid; i < 2 * stages * L::kWarps; i += L::kThreads + 32) heads[i] = -1;
  ring.start();
  begin(ranks);

  if (warp == L::kWarps) {
    if (tid == NT) ring.run();
  } else if (warp == L::kWarps + 1) {
    auto prepare = [&](int64_t r) {
      const int64_t t = ring.first + r * ring.step;
      if (t >= g.T) return;
      const int par = r & 1;
      const RowPart<T> p(logits + t * g.ldz, V, rank, ranks);
      ListRegs list;
      list_row(g, t, p, false, lists[par], list);
      if (tail) mark_listed<T, L>(p, list, V, marks[par], heads + par * stages * L::kWarps);
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&hand.ready[par]);
    };
    prepare(0);
    prepare(1);
    int64_t r = 0;
    for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
      const int par = r & 1;
      const uint32_t phase = (r >> 1) & 1;
      if (rank == 0) {
        if (!__all_sync(~0u, p24_wait(&hand.stats[par], phase, &ring_sh.abort, status))) break;
        store_loss(g, t, lists[par], hand.row[par]);
      }
      // Once a wait of this CTA has run out, a list may not have been used up: no other is chained to it.
      const bool freed = p24_wait(&hand.freed[par], phase, &ring_sh.abort, status) &&
                         *const_cast<volatile int*>(&ring_sh.abort) == 0;
      if (!__all_sync(~0u, freed)) break;
      prepare(r + 2);
    }
  } else {
    float edge = load_edge(RowPart<T>(logits + ring.first * g.ldz, V, rank, ranks));
    int64_t r = 0;
    for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
      const int par = r & 1;
      const RowPart<T> p(logits + t * g.ldz, V, rank, ranks);
      const int vecs = p.hi - p.lo;
      const ListShared& sh = lists[par];
      const Marks& mk = marks[par];
      int* head = heads + par * stages * L::kWarps;
      // false where the wait ran out: nothing of the list is used then, it may be half written
      const bool listed = __all_sync(~0u, p24_wait(&hand.ready[par], (r >> 1) & 1, &ring_sh.abort, status));

      // one pass over the row: sums (tail: off the list)
      Walk<false> w, w1;
      if (tid < p.edges) {
        if (kTwo) w1.add_one(edge, kLog2e);
        if (!tail || !((mk.edges >> tid) & 1u)) w.add_one(edge, c);
      }
      const float edge_here = edge;
      if (t + ring.step < g.T) edge = load_edge(RowPart<T>(logits + (t + ring.step) * g.ldz, V, rank, ranks));
      for (int at = 0; at < stages; ++at) {
        uint4* data = ring.wait();
        const int n = vecs - at * L::kStage;
        uint32_t mr = Vec<T>::kFill;
        if (kTwo) {
          R::each(data, n, [&](const uint4& x, int) { mr = max_vec<T>(mr, x); });
          w1.raise(max_of<T>(mr), kLog2e);
          R::each(data, n, [&](const uint4& x, int) { w1.template add<T>(x, kLog2e); });
          if (tail) mr = Vec<T>::kFill;
        }
        if (tail) {
          // the listed elements become -inf in the stage: the sums off the list have their own maximum
          const int j = listed ? head[at * L::kWarps + warp] : -1;
          if (j >= 0) {
            __syncwarp();
            if ((tid & 31) == 0) head[at * L::kWarps + warp] = -1;  // for the row after the next
            chain_walk(j, mk.next, kTopMax, [&](int e) {
              if ((tid & 31) == mk.lane[e])
                *reinterpret_cast<T*>(reinterpret_cast<char*>(data - tid) + mk.byte[e]) = static_cast<T>(ninf());
            });
            fence_proxy_async_smem();  // the next copy into this stage comes after these stores
            __syncwarp();
          }
        }
        if (!kTwo || tail) R::each(data, n, [&](const uint4& x, int) { mr = max_vec<T>(mr, x); });
        w.raise(max_of<T>(mr), c);
        R::each(data, n, [&](const uint4& x, int) { w.template add<T>(x, c); });
        ring.release();
      }

      Sums rest = w.sums(), one = w1.sums();
      row_join<false, kTwo, NT>(rest, c, one, kLog2e, joins, r, rank, ranks, &ring_sh.abort, status);
      const Sums all = tail ? join(rest, Sums{sh.top, sh.s_list, 0.f}, c) : rest;
      RowStats st;
      st.m = all.s == 0.f ? ninf() : all.m;
      st.ls = all.s == 0.f ? ninf() : logf(all.s);
      st.rest_m = rest.m;
      st.rest_ls = !tail ? 0.f : rest.s == 0.f ? ninf() : logf(rest.s);
      st.lr = !tail ? 0.f : rest.s == 0.f ? ninf() : st.rest_ls + (rest.m - st.m) / tau;  // at the reference m
      st.l1 = !g.labels ? 0.f : !kTwo ? st.ls : one.s == 0.f ? ninf() : logf(one.s);
      if (tid == 0) {
        hand.row[par] = st;
        mbar_arrive(&hand.stats[par]);
      }
      if constexpr (kGrad) {
        T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
        const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(p.row) & 15u);
        const RowGrad rg = row_grad(sh, kTwo, tau, st);
        if (tid < p.edges) out[p.edge_pos(tid)] = static_cast<T>(rg.off.template one<kTwo>(edge_here));
        store_row<T, kTwo, R>(ring, out, aligned, p, stages, rg.off);
        walk_sync<NT>();
        if (listed) store_listed<T, kTwo, NT>(out, p, sh, K, rg);
      }
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&hand.freed[par]);
    }
    end(ranks, &ring_sh.abort);
  }
}

// ln p_r from which the saved statistics give the bucket's gradient: the softmax off the list comes
// out of lr with an error of 4u |lr|, here 2^-16, as much as a sum of a long row may have. Rows
// below take their sum off the list again: a whole batch of them, 2048 x 131072, 620 us instead of 173.
constexpr float kFar = -64.f;

// This CTA's sums off the list over its share of a row, from memory: all walking threads. hit: which
// vectors (modulo 32 kHit) hold a listed element; the list is searched for those alone (with 32 words
// nearly every warp searched it: 2000 us for that batch).
constexpr int kHit = 256;
template <typename T, int NT>
__device__ __noinline__ Sums sums_off_list(const T* row, int V, int part, int parts, const ListShared& sh, int K, float c,
                                           uint32_t (&hit)[kHit]) {
  constexpr int N = Vec<T>::N;
  const RowPart<T> p(row, V, part, parts);
  const int tid = threadIdx.x;
  for (int i = tid; i < kHit; i += NT) hit[i] = 0;
  walk_sync<NT>();
  for (int j = tid; j < K; j += NT) {
    const int i = sh.idx[j];
    if (i < p.head || i >= p.tail0) continue;
    const int v = (i - p.head) / N;
    atomicOr(&hit[v / 32 % kHit], 1u << (v & 31));
  }
  walk_sync<NT>();
  Walk<false> w;
  if (tid < p.edges) {
    const int pos = p.edge_pos(tid);
    bool listed = false;
    for (int j = 0; j < K; ++j) listed |= sh.idx[j] == pos;
    if (!listed) w.add_one(to_f32(p.row[pos]), c);
  }
#pragma unroll 1
  for (int v = p.lo + tid; v < p.hi; v += NT) {
    uint4 x = p.body[v];
    if (hit[v / 32 % kHit] >> (v & 31) & 1u) {
      uint32_t r[4] = {x.x, x.y, x.z, x.w};
      const int i0 = p.vec_pos(v);
#pragma unroll 1
      for (int j = 0; j < K; ++j) {
        const int e = sh.idx[j] - i0;
        if (e < 0 || e >= N) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (e != i) continue;
          if constexpr (sizeof(T) == 2)
            r[i / 2] = (i & 1) ? (r[i / 2] & 0xffffu) | 0xff800000u : (r[i / 2] & 0xffff0000u) | 0xff80u;
          else
            r[i] = Vec<T>::kFill;
        }
      }
      x = make_uint4(r[0], r[1], r[2], r[3]);
    }
    w.raise(max_of<T>(max_vec<T>(Vec<T>::kFill, x)), c);
    w.template add<T>(x, c);
  }
  return w.sums();
}

// The gradient from saved statistics. The CTA's last warp fills the ring, the others walk the rows.
// A row is split in `parts`. kBucket: over a cluster, whose CTAs join the sums off the list of a row
// for which the statistics do not do.
template <typename T, bool kTwo, bool kBucket, typename L>
__global__ void __launch_bounds__(L::kThreads, L::kCtas) distill_bwd_kernel(const p24_distill_args g, int parts, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT, N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 ring_data[];
  __shared__ RingShared<L::S> ring_sh;
  __shared__ ListShared lists[2];
  __shared__ JoinShared joins;  // kBucket
  __shared__ uint32_t hit[kHit];  // kBucket
  const int tid = threadIdx.x, warp = tid >> 5, V = static_cast<int>(g.V), K = static_cast<int>(g.K);
  const int part = blockIdx.x % parts;
  const float tau = g.temperature;
  const T* logits = static_cast<const T*>(g.logits);
  const int stages = row_stages(V / N, parts, L::kStage);
  R ring{logits, g.ldz, blockIdx.x / parts, gridDim.x / parts, g.T, V, part, parts, stages, 1, ring_data, &ring_sh, status};
  if (kBucket && tid == 0) join_init(joins, parts);
  ring.start();
  begin(kBucket ? parts : 1);
  if (tid >= NT) {
    if (tid == NT) ring.run();
    return;
  }
  float edge = load_edge(RowPart<T>(logits + ring.first * g.ldz, V, part, parts));
  int64_t r = 0, joined = 0;
  for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
    const RowPart<T> p(logits + t * g.ldz, V, part, parts);
    ListShared& sh = lists[r & 1];
    RowStats st{g.stats[4 * t], g.stats[4 * t + 1], g.stats[4 * t + 2], g.stats[4 * t + 3], 0.f, 0.f};
    if (warp == 0) {
      ListRegs list;
      list_row(g, t, p, true, sh, list);  // another part's logits are being overwritten, in place
    }
    walk_sync<NT>();
    if constexpr (kBucket) {
      st.rest_m = st.m;
      st.rest_ls = st.lr;
      // the same in every CTA of the cluster: from the statistics and the list
      if (sh.q_rest > 0.f && st.ls != ninf() && !(st.lr - st.ls >= kFar)) {
        const float c = kLog2e / tau;
        Sums rest = sums_off_list<T, NT>(p.row, V, part, parts, sh, K, c, hit), unused{0.f, 0.f, 0.f};
        row_join<false, false, NT>(rest, c, unused, c, joins, joined++, part, parts, &ring_sh.abort, status);
        st.rest_m = rest.m;
        st.rest_ls = rest.s == 0.f ? ninf() : logf(rest.s);
      }
    }
    T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(p.row) & 15u);
    const RowGrad rg = row_grad(sh, kTwo, tau, st);
    if (tid < p.edges) out[p.edge_pos(tid)] = static_cast<T>(rg.off.template one<kTwo>(edge));
    if (t + ring.step < g.T) edge = load_edge(RowPart<T>(logits + (t + ring.step) * g.ldz, V, part, parts));
    store_row<T, kTwo, R>(ring, out, aligned, p, stages, rg.off);
    walk_sync<NT>();
    store_listed<T, kTwo, NT>(out, p, sh, K, rg);
  }
  if constexpr (kBucket) end(parts, &ring_sh.abort);
}

template <typename T, bool kTwo, bool kGrad>
cudaError_t launch_distill_as(const p24_distill_args& g, int* status, cudaStream_t s) {
  using L = std::conditional_t<kGrad, Step, Loss>;
  const int64_t vecs = g.V / Vec<T>::N;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  auto smem = [&](auto layout, int ranks) {
    using M = decltype(layout);
    return static_cast<size_t>(M::kRing + (tail ? 2 * row_stages(vecs, ranks, M::kStage) * M::kWarps * 4 : 0));
  };
  if (vecs <= kShortRow && g.T > sm_count())
    return launch_rows(distill_kernel<T, kTwo, kGrad, Short>, Short::kThreads + 32, g.T, 1, smem(Short(), 1), s, g, status);
  int ranks = 1;
  // The rows in flight stay in L2 (129 MB, outputs among them) until they come the second time: with
  // 61 MB of them every second visit hit, with 80 MB a quarter went to memory, with 160 MB nearly all.
  constexpr int64_t kL2Rows = 64 << 20;
  while (kGrad && ranks < kMaxRanks && std::min<int64_t>(g.T, sm_count() * L::kCtas / ranks) * vecs * 16 > kL2Rows) ranks *= 2;
  // 800 vectors a CTA: loss of 256 x 131072 14.4 us over 2 CTAs a row, 17.7 whole, 18.3 over 4; loss and
  // gradient of 64 x 32000 6.3 over 4, 7.4 whole, 9.2 over 8. Nothing in it knows of rows that fill the
  // memory's rate whole: of 256 x 131072, 32.6 over 4 and 29.1 whole; loss of 400 x 131072 24.0 over 2, 21.4 whole.
  ranks = std::max(ranks, row_split(g.T, vecs, sm_count() * L::kCtas, kMaxRanks, 800));
  return launch_rows(distill_kernel<T, kTwo, kGrad, L>, L::kThreads + 32, g.T, ranks, smem(L(), ranks), s, g, status);
}

template <typename T, bool kTwo>
cudaError_t launch_distill_bwd_as(const p24_distill_args& g, int* status, cudaStream_t s) {
  const int64_t vecs = g.V / Vec<T>::N;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  if (vecs <= kShortRow)
    return launch_parts(tail ? distill_bwd_kernel<T, kTwo, true, ShortGrad> : distill_bwd_kernel<T, kTwo, false, ShortGrad>,
                        ShortGrad::kThreads, g.T, 1, ShortGrad::kRing, s, g, 1, status);
  // 512 vectors a CTA: 64 x 32000 4.4 us over 4 CTAs a row, 5.9 whole; 256 x 131072 19.9 over 2, 21.6 whole,
  // 22.7 over 4; 1200 x 50257 41.8 whole, 46.0 over 2; 900 x 32000 20.9 whole, 20.5 over 2.
  const int parts = row_split(g.T, vecs, sm_count() * Grad::kCtas, tail ? kMaxRanks : 64, 512);
  if (tail)
    return launch_rows(distill_bwd_kernel<T, kTwo, true, Grad>, Grad::kThreads, g.T, parts, Grad::kRing, s, g, parts, status);
  return launch_parts(distill_bwd_kernel<T, kTwo, false, Grad>, Grad::kThreads, g.T, parts, Grad::kRing, s, g, parts, status);
}

template <typename T>
cudaError_t launch_distill_type(const p24_distill_args& g, bool bwd, int* st, cudaStream_t s) {
  const bool two = g.labels && g.temperature != 1.f;
  if (bwd) return two ? launch_distill_bwd_as<T, true>(g, st, s) : launch_distill_bwd_as<T, false>(g, st, s);
  if (g.dlogits) return two ? launch_distill_as<T, true, true>(g, st, s) : launch_distill_as<T, false, true>(g, st, s);
  return two ? launch_distill_as<T, true, false>(g, st, s) : launch_distill_as<T, false, false>(g, st, s);
}

}  // namespace

cudaError_t launch_distill(const p24_distill_args& g, int* status, cudaStream_t s) {
  return g.dtype == P24_BF16 ? launch_distill_type<__nv_bfloat16>(g, false, status, s)
                             : launch_distill_type<float>(g, false, status, s);
}

cudaError_t launch_distill_bwd(const p24_distill_args& g, int* status, cudaStream_t s) {
  return g.dtype == P24_BF16 ? launch_distill_type<__nv_bfloat16>(g, true, status, s)
                             : launch_distill_type<float>(g, true, status, s);
}

}  // namespace p24
