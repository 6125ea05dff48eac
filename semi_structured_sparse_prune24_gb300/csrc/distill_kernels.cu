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
//                      when the list holds nearly everything): a bit per element, one byte
//                      per vector, says which ones. The gradient follows from the
//                      row's second way through the ring (from L2); the listed columns and the label are then stored again
//                      with their own terms.
//  distill_bwd_kernel  the gradient alone, elementwise from the saved statistics.
//
// Bound: HBM, one read of the logits (and one write of the gradient).
#include <algorithm>
#include <type_traits>

#include "head_rows.cuh"

namespace p24 {
namespace {

// ---------------------------------------------------------------- the teacher's list
// One row's list in shared memory; two of them take turns, so that a row's is not overwritten
// while the last gradient elements of the row before are stored.
struct ListShared {
  int idx[kTopMax];   // column, -1 for an absent entry
  float z[kTopMax];   // the student's logit there
  float q[kTopMax];   // the teacher's probability
  float q_sum, q_rest;
  float top, s_list;  // the listed logits' maximum and their sum of exp((z - top) / tau)
  int label_listed;
};

constexpr int kPerLane = kTopMax / 32;

// A warp's copy of a list, entry j in lane j % 32, slot j / 32.
struct ListRegs {
  int idx[kPerLane];
  float val[kPerLane];

  __device__ __forceinline__ void load(const p24_distill_args& g, int64_t t, bool on) {
    const int K = static_cast<int>(g.K), lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int j = lane + 32 * i;
      idx[i] = -1;
      val[i] = ninf();
      if (on && j < K) {
        idx[i] = g.top_idx[t * K + j];
        val[i] = g.top_val[t * K + j];
      }
    }
  }
};

// What a warp needs of a row's list: lane j % 32 has entry j in slot j / 32.
struct ListZ {
  float z[kPerLane];
  // own: only the elements of this CTA. Read before an in-place gradient overwrites them.
  template <typename T>
  __device__ __forceinline__ void load(const RowPart<T>& p, bool own, const ListRegs& r, int V) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      z[i] = r.idx[i] >= 0 && r.idx[i] < V && (!own || p.owns(r.idx[i])) ? to_f32(p.row[r.idx[i]]) : ninf();
  }
};

// The list with the teacher's probabilities, into shared memory: warp 0.
__device__ __forceinline__ void list_row(const p24_distill_args& g, const ListRegs& r, const ListZ& rz, int label,
                                         ListShared& sh) {
  const int K = static_cast<int>(g.K), V = static_cast<int>(g.V), lane = threadIdx.x & 31;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  const float tau = g.temperature;
  float q[kPerLane];
  float vtop = ninf(), ztop = ninf();
  bool listed = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const bool on = r.idx[i] >= 0 && r.idx[i] < V;
    q[i] = on ? r.val[i] : ninf();
    vtop = fmaxf(vtop, q[i]);
    ztop = fmaxf(ztop, rz.z[i]);
    listed |= on && r.idx[i] == label;
  }
  vtop = warp_max(vtop);
  ztop = warp_max(ztop);
  float sum = 0.f, s = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const float x = q[i], z = rz.z[i];
    // absent: 0; a NaN stays one; the list's softmax at the temperature, or the probabilities as they are
    q[i] = x != x ? x : x == ninf() ? 0.f : expf(tail ? x : (x - vtop) / tau);
    sum += q[i];
    if (ztop > ninf() || z != z) s += ex2(floored(z - ztop) * (kLog2e / tau));
  }
  sum = warp_sum(sum);
  s = warp_sum(s);
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int j = lane + 32 * i;
    if (j < K) {
      sh.idx[j] = r.idx[i] >= 0 && r.idx[i] < V ? r.idx[i] : -1;
      sh.z[j] = rz.z[i];
      sh.q[j] = !tail && sum != 0.f ? q[i] / sum : q[i];
    }
  }
  listed = __any_sync(~0u, listed);
  if (lane == 0) {
    sh.q_rest = tail ? fmaxf(1.f - sum, 0.f) : 0.f;
    sh.q_sum = tail ? sum : sum != 0.f ? 1.f : 0.f;
    sh.top = ztop;
    sh.s_list = s;
    sh.label_listed = listed;
  }
}

// The label and the weights of a row.
struct RowArgs {
  int label;
  float dkl, dce;

  __device__ __forceinline__ void load(const p24_distill_args& g, int64_t t) {
    label = g.labels ? g.labels[t] : -1;
    dkl = g.dkl ? g.dkl[t] : 0.f;
    dce = g.dce ? g.dce[t] : 0.f;
  }
  __device__ __forceinline__ void check(int V) {
    if (label < 0 || label >= V) label = -1, dce = 0.f;
  }
};

// A row's gradient: its terms off the list and on it, the factor on q and the label's.
struct RowGrad {
  Terms off, on;
  float wq, wl;
};
// dkl, dce: the row's weights. m, ls, lr, l1: its statistics.
__device__ __forceinline__ RowGrad row_grad(const ListShared& sh, bool two, float tau, float m, float ls, float lr,
                                            float l1, float dkl, float dce) {
  RowGrad r;
  // a row with nothing above -inf: all terms 0
  const bool none = ls == ninf();
  if (none) m = ls = l1 = dkl = dce = 0.f;
  const float q_rest = lr == ninf() ? 0.f : sh.q_rest;  // a bucket in which the student can have nothing is dropped
  r.wq = dkl / tau;
  r.wl = dce;
  r.on.m = m, r.on.c = kLog2e / tau, r.on.off = -ls * kLog2e, r.on.off1 = -l1 * kLog2e;
  r.on.w = r.wq * (sh.q_sum + q_rest);
  r.on.w1 = dce;
  r.off = r.on;
  if (q_rest > 0.f) {
    // Q p - q_r p / p_r = (Q p_r - q_r) exp(x - lr), where neither p nor p_r alone may underflow
    const float p_rest = expf(lr - ls);
    r.off.off = -lr * kLog2e;
    r.off.w = r.wq * ((sh.q_sum + q_rest) * p_rest - q_rest);
    if (!two) r.off.w += dce * p_rest;
  } else if (!two) {
    r.off.w += dce;  // one temperature: the label's softmax is p
  }
  if (!two) r.on.w += dce;
  return r;
}

// The gradient's terms off the list over the stages of a row, whose first is stage `from` of the row's sequence.
template <typename T, bool kTwo, typename R>
__device__ __forceinline__ void store_row(R& ring, int64_t r, int from, T* out, bool aligned, const RowPart<T>& p, int stages,
                                          const Terms& terms) {
  constexpr int N = Vec<T>::N, NT = R::kThreads;
  for (int at = 0; at < stages; ++at) {
    const uint4* data = ring.wait();
    const int v0 = p.lo + at * R::kStage + static_cast<int>(threadIdx.x);
    R::each(data, p.hi - p.lo - at * R::kStage, [&](const uint4& x, int u) {
      F2 y[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) y[j] = terms.template two<kTwo>(pair<T>(x, j));
      store_vec(out, p.vec_pos(v0 + u * NT), aligned, pack_vec<T>(y));
    });
    ring.release(r, from + at);
  }
}

// The listed columns and the label, stored after the rest of the row (and a barrier).
template <typename T, bool kTwo, int NT>
__device__ __forceinline__ void store_listed(T* out, const RowPart<T>& p, const ListShared& sh, int K, int label,
                                             float z_label, const RowGrad& rg) {
  for (int j = threadIdx.x; j <= K; j += NT) {
    const int i = j < K ? sh.idx[j] : (sh.label_listed ? -1 : label);
    if (i < 0 || !p.owns(i)) continue;
    float y = j < K ? rg.on.template one<kTwo>(sh.z[j]) - rg.wq * sh.q[j] : rg.off.template one<kTwo>(z_label);
    if (i == label) y -= rg.wl;
    out[i] = static_cast<T>(y);
  }
}

using Loss = Layout<128, 8, 4, 3>;
using Step = Layout<256, 3, 4, 4>;
using Grad = Layout<256, 4, 4, 3>;
using Short = Layout<128, 8, 2, 4>;  // rows of up to kShortRow vectors
constexpr int kShortRow = 1024;

// The listed elements of a CTA's share, a byte per vector: byte u of word [stage][thread] is for
// vector u of that thread's stage.
template <int SV>
using MaskWord = std::conditional_t<SV == 4, uint32_t, uint16_t>;

template <typename T, typename L>
__device__ __forceinline__ void mark_listed(const RowPart<T>& p, const ListRegs& r, int V, MaskWord<L::SV>* listed,
                                            uint32_t* listed_edges) {
  constexpr int N = Vec<T>::N;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int at = r.idx[i];
    if (at < 0 || at >= V || !p.owns(at)) continue;
    if (at >= p.head && at < p.tail0) {
      const int v = (at - p.head) / N - p.lo, bit = (at - p.head) % N;
      const int byte = (v / L::kStage * L::NT + v % L::NT) * L::SV + v % L::kStage / L::NT;
      atomicOr(reinterpret_cast<uint32_t*>(listed) + (byte >> 2), 1u << (8 * (byte & 3) + bit));
    } else {
      atomicOr(listed_edges, 1u << (at < p.head ? at : p.head + at - p.tail0));
    }
  }
}

// kGrad: with the gradient. kTwo: the label's softmax (temperature 1) differs from the list's.
template <typename T, bool kTwo, bool kGrad, typename L>
__global__ void __launch_bounds__(L::NT, L::kCtas) distill_kernel(const p24_distill_args g, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT, N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 ring_data[];
  auto* listed = reinterpret_cast<MaskWord<L::SV>*>(reinterpret_cast<char*>(ring_data) + L::kRing);  // tail
  __shared__ RingShared<L::S> ring_sh;
  __shared__ JoinShared joins, joins1;
  __shared__ ListShared lists[2];
  __shared__ uint32_t listed_edges;
  const int tid = threadIdx.x, warp = tid >> 5, V = static_cast<int>(g.V), K = static_cast<int>(g.K);
  const int ranks = cluster_ranks(), rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  const float tau = g.temperature, c = kLog2e / tau;
  const T* logits = static_cast<const T*>(g.logits);
  const int stages = row_stages(V / N, ranks, L::kStage);
  R ring{logits, g.ldz, blockIdx.x / ranks, gridDim.x / ranks, g.T, V, rank, ranks, stages, kGrad ? 2 : 1,
         ring_data, &ring_sh, status};
  ring.start();
  RowPart<T> p(logits + ring.first * g.ldz, V, rank, ranks);
  float edge = load_edge(p, true);
  RowArgs args;
  args.load(g, ring.first);
  ListRegs list;
  if (warp == 0) list.load(g, ring.first, true);
  if (tail) {
    for (int i = tid; i < stages * NT; i += NT) listed[i] = 0;
    if (tid == 0) listed_edges = 0;
    __syncthreads();
    if (warp == 0) mark_listed<T, L>(p, list, V, listed, &listed_edges);
    __syncthreads();
  }
  if (ranks > 1) cluster_barrier();  // every CTA runs before another writes to its shared memory

  int64_t r = 0;
  for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
    const int par = r & 1, vecs = p.hi - p.lo;
    const bool more = t + ring.step < g.T;
    const RowPart<T> next(logits + (more ? t + ring.step : t) * g.ldz, V, rank, ranks);
    ListShared& sh = lists[par];
    RowArgs now = args;
    now.check(V);
    const float z_label = now.label >= 0 ? to_f32(p.row[now.label]) : 0.f;  // before an in-place gradient overwrites it
    if (more) args.load(g, t + ring.step);
    ListZ list_z;
    if (warp == 0) list_z.load(p, false, list, V);

    // one pass over the row: sums (tail: off the list)
    Walk<false> w, w1;
    if (tid < p.edges) {
      if (kTwo) w1.add_one(edge, kLog2e);
      if (!tail || !((listed_edges >> tid) & 1u)) w.add_one(edge, c);
    }
    const float edge_here = edge;
    edge = load_edge(next, more);
    for (int at = 0; at < stages; ++at) {
      MaskWord<L::SV> skip = 0;
      if (tail) {
        skip = listed[at * NT + tid];
        if (skip) listed[at * NT + tid] = 0;  // for the next row
      }
      const bool masked = tail && __any_sync(~0u, skip != 0);
      const uint4* data = ring.wait();
      const int n = vecs - at * L::kStage;
      uint32_t mr = Vec<T>::kFill;
      if (kTwo || !masked) R::each(data, n, [&](const uint4& x, int) { mr = max_vec<T>(mr, x); });
      if (kTwo) {
        w1.raise(max_of<T>(mr), kLog2e);
        R::each(data, n, [&](const uint4& x, int) { w1.template add<T>(x, kLog2e); });
      }
      if (masked) {  // without the listed elements: the sums off the list keep their own maximum
        auto unlisted = [&](const uint4& x, int u) { return without<T>(x, static_cast<uint32_t>(skip >> (8 * u)) & 255u); };
        mr = Vec<T>::kFill;
        R::each(data, n, [&](const uint4& x, int u) { mr = max_vec<T>(mr, unlisted(x, u)); });
        w.raise(max_of<T>(mr), c);
        R::each(data, n, [&](const uint4& x, int u) { w.template add<T>(unlisted(x, u), c); });
      } else {
        w.raise(max_of<T>(mr), c);
        R::each(data, n, [&](const uint4& x, int) { w.template add<T>(x, c); });
      }
      ring.release(r, at);
    }
    if (warp == 0) {
      list_row(g, list, list_z, now.label, sh);
      list.load(g, more ? t + ring.step : t, more);
    }

    const Sums rest = row_join<false, NT>(w.sums(), c, joins, par, rank, ranks);
    Sums one{0.f, 0.f, 0.f};
    if (kTwo) one = row_join<false, NT>(w1.sums(), kLog2e, joins1, par, rank, ranks);
    const Sums all = tail ? join(rest, Sums{sh.top, sh.s_list, 0.f}, c) : rest;
    const float m = all.s == 0.f ? ninf() : all.m;
    const float ls = all.s == 0.f ? ninf() : logf(all.s);
    // off the list, at the reference m
    float lr = 0.f;
    if (tail) lr = rest.s == 0.f ? ninf() : logf(rest.s) + (rest.m - m) / tau;
    const float l1 = !g.labels ? 0.f : !kTwo ? ls : one.s == 0.f ? ninf() : logf(one.s);
    if (warp == 0) {
      if (rank == 0) {
        float kl = 0.f;
        for (int j = tid; j < K; j += 32) {
          const float q = sh.q[j];
          const float lp = all.s == 0.f ? ninf() : (sh.z[j] - m) / tau - ls;
          if (q != 0.f) kl += q * (logf(q) - lp);
        }
        kl = warp_sum(kl);
        if (tid == 0) {
          const float qr = lr == ninf() ? 0.f : sh.q_rest;
          if (qr > 0.f) kl += qr * (logf(qr) - (lr - ls));
          g.kl[t] = kl;
          if (g.ce) g.ce[t] = now.label < 0 ? 0.f : all.s == 0.f ? -ninf() : l1 - (z_label - m);
          if (g.stats) {
            g.stats[4 * t] = m;
            g.stats[4 * t + 1] = ls;
            g.stats[4 * t + 2] = lr;
            g.stats[4 * t + 3] = l1;
          }
        }
      }
      if (tail) {  // the next row's listed elements: every thread has read and cleared this row's
        if (tid == 0) listed_edges = 0;
        __syncwarp();
        mark_listed<T, L>(next, list, V, listed, &listed_edges);
      }
    }
    if constexpr (kGrad) {
      T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
      const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(p.row) & 15u);
      const RowGrad rg = row_grad(sh, kTwo, tau, m, ls, lr, l1, now.dkl, now.dce);
      if (tid < p.edges) out[p.edge_pos(tid)] = static_cast<T>(rg.off.template one<kTwo>(edge_here));
      store_row<T, kTwo, R>(ring, r, stages, out, aligned, p, stages, rg.off);
    }
    if (kGrad || tail) __syncthreads();
    if (kGrad)
      store_listed<T, kTwo, NT>(static_cast<T*>(g.dlogits) + t * g.ldd, p, sh, K, now.label, z_label,
                                row_grad(sh, kTwo, tau, m, ls, lr, l1, now.dkl, now.dce));
    p = next;
  }
  ring.finish();
}

template <typename T, bool kTwo, typename L>
__global__ void __launch_bounds__(L::NT, L::kCtas) distill_bwd_kernel(const p24_distill_args g, int parts, int* status) {
  using R = Ring<T, L>;
  constexpr int NT = L::NT, N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 ring_data[];
  __shared__ RingShared<L::S> ring_sh;
  __shared__ ListShared lists[2];
  const int tid = threadIdx.x, warp = tid >> 5, V = static_cast<int>(g.V), K = static_cast<int>(g.K);
  const int part = blockIdx.x % parts;
  const float tau = g.temperature;
  const T* logits = static_cast<const T*>(g.logits);
  const int stages = row_stages(V / N, parts, L::kStage);
  R ring{logits, g.ldz, blockIdx.x / parts, gridDim.x / parts, g.T, V, part, parts, stages, 1, ring_data, &ring_sh, status};
  ring.start();
  struct Stats {
    float m, ls, lr, l1;
  };
  auto stats_of = [&](int64_t t) { return Stats{g.stats[4 * t], g.stats[4 * t + 1], g.stats[4 * t + 2], g.stats[4 * t + 3]}; };
  RowPart<T> p(logits + ring.first * g.ldz, V, part, parts);
  float edge = load_edge(p, true);
  RowArgs args;
  args.load(g, ring.first);
  Stats stats = stats_of(ring.first);
  ListRegs list;
  if (warp == 0) list.load(g, ring.first, true);
  int64_t r = 0;
  for (int64_t t = ring.first; t < g.T; t += ring.step, ++r) {
    const bool more = t + ring.step < g.T;
    const RowPart<T> next(logits + (more ? t + ring.step : t) * g.ldz, V, part, parts);
    ListShared& sh = lists[r & 1];
    RowArgs now = args;
    now.check(V);
    const Stats st = stats;
    // read before an in-place gradient overwrites them; another part's are not used here
    const float z_label = now.label >= 0 && p.owns(now.label) ? to_f32(p.row[now.label]) : 0.f;
    if (warp == 0) {
      ListZ list_z;
      list_z.load(p, true, list, V);
      list_row(g, list, list_z, now.label, sh);
      list.load(g, more ? t + ring.step : t, more);
    }
    if (more) {
      args.load(g, t + ring.step);
      stats = stats_of(t + ring.step);
    }
    __syncthreads();
    T* out = static_cast<T*>(g.dlogits) + t * g.ldd;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15u) == (reinterpret_cast<uintptr_t>(p.row) & 15u);
    const RowGrad rg = row_grad(sh, kTwo, tau, st.m, st.ls, st.lr, st.l1, now.dkl, now.dce);
    if (tid < p.edges) out[p.edge_pos(tid)] = static_cast<T>(rg.off.template one<kTwo>(edge));
    edge = load_edge(next, more);
    store_row<T, kTwo, R>(ring, r, 0, out, aligned, p, stages, rg.off);
    __syncthreads();
    store_listed<T, kTwo, NT>(out, p, sh, K, now.label, z_label, rg);
    p = next;
  }
  ring.finish();
}

template <typename T, bool kTwo, bool kGrad>
cudaError_t launch_distill_as(const p24_distill_args& g, int* status, cudaStream_t s) {
  using L = std::conditional_t<kGrad, Step, Loss>;
  const int64_t vecs = g.V / Vec<T>::N;
  const bool tail = (g.flags & P24_DISTILL_TAIL) != 0;
  auto smem = [&](auto layout, int ranks) {
    using M = decltype(layout);
    return static_cast<size_t>(M::kRing + (tail ? row_stages(vecs, ranks, M::kStage) * M::NT * M::SV : 0));
  };
  if (vecs <= kShortRow && g.T > sm_count())
    return launch_rows(distill_kernel<T, kTwo, kGrad, Short>, Short::NT, g.T, 1, smem(Short(), 1), s, g, status);
  int ranks = 1;
  while (ranks < kMaxRanks && smem(L(), ranks) > 200 * 1024) ranks *= 2;  // the mask of a very long row
  ranks = row_ranks<L>(ranks, g.T, vecs);
  return launch_rows(distill_kernel<T, kTwo, kGrad, L>, L::NT, g.T, ranks, smem(L(), ranks), s, g, status);
}

template <typename T, bool kTwo>
cudaError_t launch_distill_bwd_as(const p24_distill_args& g, int* status, cudaStream_t s) {
  const int64_t vecs = g.V / Vec<T>::N;
  if (vecs <= kShortRow)
    return launch_parts(distill_bwd_kernel<T, kTwo, Short>, Short::NT, g.T, 1, Short::kRing, s, g, 1, status);
  const int parts = row_parts<Grad>(g.T, vecs);
  return launch_parts(distill_bwd_kernel<T, kTwo, Grad>, Grad::NT, g.T, parts, Grad::kRing, s, g, parts, status);
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
