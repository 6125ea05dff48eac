"""GPU parity of the language-model head's row operators (p24_token_logprobs,
p24_distill_topk and their gradients) against the fp64 oracle (oracle/head_oracle.py).

Tolerances, derived for u = 2^-24 and x = (z - m) / tau:
  * x takes three roundings, so exp(x) is off by at most 3u|x| + 4u relative (2^-22 for the
    exponential). Weighted by p that is 3u E|x| + 4u, and E|x| <= ln V <= 12.
  * The sum of positive terms adds at most u per addition on a term's way: at most
    V / 512 + 8 in a thread, two roundings for each rise of the running maximum (fewer than
    64 are allowed for), 5 across a warp and 16 across the CTA. Together
        e_s = (256 + V / 512) u      relative on s, absolute on ln s.
  * log probabilities, CE and KL:  e_s + 8u |value| + 8u |ln s|, KL with the list's own
    roundings: 2 e_s + 16u sum q (|ln q| + |ln p|).
  * the entropy's weighted sum carries the same errors times |x|: e_s (2 + ln V).
  * the bucket's 1 - sum q is off by at most 64u absolute (K <= 128 terms of sum <= 1,
    exp 2u): relative 64u / q_r wherever q_r enters.
  * gradients: each p is off by (e_s + 4u|x| + 16u) relative; bf16 outputs are then rounded
    (2^-9 relative, and the fp32 error may move a rounding: 2^-8).
Positions are compared exactly: the order of the logits is exact.
"""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def e_s(V):
    return (256 + V / 512) * U


def logits(T, V, dtype, seed, sigma=2.5, pad=0, peak=True):
    """[T, V] logits with a likely token per row, as a view with row stride V + pad."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(T, V)) * sigma
    if peak:
        z[np.arange(T), rng.integers(0, V, T)] += rng.random(T) * 12
    full = torch.full((T, V + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :V] = torch.as_tensor(z, device="cuda").to(dtype)
    return full[:, :V], rng


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda").to(dtype)


def close(got, want, bound, name):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), name
    bad = np.abs(got - want)[fin] > np.broadcast_to(bound, want.shape)[fin]
    assert not bad.any(), (name, int(bad.sum()), got[fin][bad][:4], want[fin][bad][:4],
                           np.broadcast_to(bound, want.shape)[fin][bad][:4])


def check_score(P, z, tokens, k, tau, ent=True):
    T, V = z.shape
    o = P.p24_token_logprobs(z, None if tokens is None else dev(tokens, torch.int32), k=k, temperature=tau, entropy=ent)
    ref = HO.token_logprobs(f64(z), tokens, k, tau)
    ls = np.abs(ref["stats"][:, 1])
    ls = np.where(np.isfinite(ls), ls, 0)
    base = e_s(V) + 8 * U * ls
    finite = lambda a: np.where(np.isfinite(a), np.abs(a), 0)  # noqa: E731
    if tokens is not None:
        close(o["logp"], ref["logp"], base + 8 * U * finite(ref["logp"]), "logp")
    if ent:
        close(o["entropy"], ref["entropy"], (e_s(V) + 8 * U * ls) * (2 + np.log(V)), "entropy")
    nan = np.isnan(ref["stats"][:, 0])  # a row with NaN or +inf: the maximum is not specified
    close(f64(o["stats"])[~nan, 0], ref["stats"][~nan, 0], 0, "max")
    close(o["stats"][:, 1], ref["stats"][:, 1], base, "ln s")
    if k:
        assert np.array_equal(o["top_idx"].cpu().numpy(), ref["top_idx"]), "top_idx"
        close(o["top_logp"], ref["top_logp"], base[:, None] + 8 * U * finite(ref["top_logp"]), "top_logp")
    return o, ref


# one token to long rows, odd sizes, rows off the 16-byte boundary, k from 0 past V
SCORE = [(1, 1, 1, 0), (3, 5, 8, 0), (1, 32000, 20, 0), (5, 7, 3, 1), (2, 4096, 128, 0), (33, 1001, 64, 0),
         (4, 50257, 20, 0), (2, 65537, 128, 7), (150, 4100, 5, 4), (700, 515, 2, 0), (9, 8191, 1, 3), (1, 131072, 64, 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k,pad", SCORE)
def test_score(P, dtype, T, V, k, pad):
    z, rng = logits(T, V, dtype, T * 7 + V, pad=pad)
    tokens = rng.integers(0, V, T)
    tokens[::5] = -1 if T > 1 else tokens[::5]
    check_score(P, z, tokens, k, [1.0, 0.7, 2.0][(T + V) % 3])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_score_parts(P, dtype):
    """Without tokens, without entropy, without alternatives; a token past the vocabulary."""
    z, _ = logits(6, 3001, dtype, 1)
    assert "logp" not in check_score(P, z, None, 3, 1.0, ent=False)[0]
    o, _ = check_score(P, z, np.array([0, 3000, 3001, -7, 2 ** 31 - 1, 5]), 0, 1.0)
    assert o["logp"][2:5].tolist() == [0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fill", ["equal", "steps", "ramp", "fall"])
@pytest.mark.parametrize("T", [2, 320])
def test_top_order_with_ties(P, dtype, fill, T):
    """All equal, a few distinct values, and rising or falling rows (the first or the last
    part of the row holds every alternative)."""
    V = 20011
    j = np.arange(V)
    row = {"equal": np.zeros(V), "steps": np.floor(j * 7919 % V / 2000.0), "ramp": j / 128.0, "fall": -(j // 16) / 16.0}[fill]
    z = dev(np.tile(row, (T, 1)), dtype)
    o = P.p24_token_logprobs(z, None, k=100)
    want = HO.order(f64(z[0]))[:100]
    assert (o["top_idx"].cpu().numpy() == want).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [6, 400])
@pytest.mark.parametrize("low", [float("-inf"), "lowest"])
def test_score_masked_rows(P, dtype, T, low):
    """Masks that leave 0, 1, 3, 12 or 300 entries of a row, by -inf and by the type's lowest
    value; k is larger than what most of them leave."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    z, rng = logits(T, 9001, dtype, 3)
    z = z.clone()
    tokens = rng.integers(0, 9001, T)
    for t in range(T):
        left = [0, 1, 3, 12, 300, 9001][t % 6]
        keep = rng.permutation(9001)[:left]
        if left:
            keep[0] = tokens[t]
        row = torch.full_like(z[t], low)
        row[torch.as_tensor(keep, device="cuda")] = z[t, torch.as_tensor(keep, device="cuda")]
        z[t] = row
    check_score(P, z, tokens, 20, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_score_nan_inf_and_signed_zero(P, dtype):
    z, _ = logits(6, 5003, dtype, 4, sigma=0.5, peak=False)
    z[0, 77] = float("nan")
    z[1, [5, 4000]] = float("inf")
    z[2, [9, 10]] = float("nan")
    z[2, 3] = float("inf")
    z[3] = -1
    z[3, 1000] = -0.0
    z[3, 2000] = 0.0
    z[4, 17] = float("-inf")
    check_score(P, z, np.array([0, 5, 1, 1000, 17, 3]), 8, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [1e4, -1e4])
def test_score_large_magnitudes(P, dtype, shift):
    """Large offsets: x = (z - m) / tau is formed from the difference, so nothing is lost."""
    z, rng = logits(4, 3003, dtype, 6, peak=False)
    z = (z.float() + shift).to(dtype)
    check_score(P, z, rng.integers(0, 3003, 4), 4, 0.7)


def grad_bound(V, want, p, x, weights, dtype, extra=0.0):
    """Bound on a gradient element: weights = the factor on p (its largest magnitude), extra =
    terms that do not scale with p."""
    b = weights * p * (e_s(V) + 4 * U * np.abs(np.where(np.isfinite(x), x, 0)) + 32 * U) + extra + 4 * U * np.abs(want)
    return b + (2.0 ** -8 * np.abs(want) + 1e-38 if dtype == BF else 1e-38)


BWD = [(1, 1, 0), (3, 7, 1), (5, 4099, 0), (2, 50257, 0), (130, 1000, 8), (1, 131072, 0), (400, 333, 5)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,pad", BWD)
@pytest.mark.parametrize("parts", ["both", "logp", "entropy"])
@pytest.mark.parametrize("inplace", [False, True])
def test_score_gradient(P, dtype, T, V, pad, parts, inplace):
    tau = [1.0, 0.7][T % 2]
    z, rng = logits(T, V, dtype, T + V, pad=pad)
    z[0, V // 2] = float("-inf") if V > 1 else z[0, V // 2]
    tokens = rng.integers(0, V, T)
    tokens[::7] = -1 if T > 2 else tokens[::7]
    g, h = rng.normal(size=T), rng.normal(size=T) * 0.1
    tok = dev(tokens, torch.int32)
    o = P.p24_token_logprobs(z, tok, temperature=tau)
    gz, hz = (g if parts != "entropy" else None), (h if parts != "logp" else None)
    Z = f64(z)
    out = z if inplace else None
    D = P.p24_token_logprobs_bwd(z, tok, o["stats"], None if gz is None else dev(g, F32),
                                 entropy=o["entropy"], dentropy=None if hz is None else dev(h, F32), temperature=tau,
                                 dlogits=out)
    g32, h32 = (f64(dev(a, F32)) for a in (g, h))
    ref = HO.token_logprobs_bwd(Z, tokens, None if gz is None else g32, None if hz is None else h32, tau)
    x = (Z - Z.max(1, keepdims=True)) / tau
    s = np.exp(x).sum(1, keepdims=True)
    p, lp = np.exp(x) / s, np.maximum(x - np.log(s), -200)
    H = f64(o["entropy"])[:, None]
    w = ((np.abs(g32) if gz is not None else 0 * g)[:, None] + (np.abs(h32) if hz is not None else 0 * h)[:, None]
         * (np.abs(lp) + H + 2 + np.log(V))) / tau
    close(D, ref, grad_bound(V, ref, p, x, w, dtype), "dlogits")


def test_score_gradient_empty_row_and_other_stride(P):
    """A fully masked row has gradient 0; a gradient with another alignment than the logits."""
    z, _ = logits(3, 1000, BF, 9, pad=8)
    z[1] = float("-inf")
    tok = dev(np.array([1, 2, 3]), torch.int32)
    o = P.p24_token_logprobs(z, tok)
    full = torch.full((3, 1003), 7.0, dtype=BF, device="cuda")
    g = dev(np.ones(3), F32)
    P.p24_token_logprobs_bwd(z, tok, o["stats"], g, entropy=o["entropy"], dentropy=g, dlogits=full[:, 1:1001])
    dense = P.p24_token_logprobs_bwd(z, tok, o["stats"], g, entropy=o["entropy"], dentropy=g)
    assert torch.equal(full[:, 1:1001], dense) and not dense[1].any()
    assert (full[:, 0] == 7).all() and (full[:, 1001:] == 7).all()


def teacher_list(rng, T, V, K, mass=0.9):
    """K distinct columns a row, falling log probabilities of total `mass`, some entries absent."""
    idx = np.stack([rng.permutation(V)[:K] if K <= V else np.r_[rng.permutation(V), np.full(K - V, -1)]
                    for _ in range(T)]).reshape(T, K).astype(np.int64)
    val = np.log(rng.dirichlet(np.ones(max(K, 1)), size=T)[:, :K] * mass + 1e-6)
    for t in range(T):
        if t % 4 == 1:
            idx[t, K // 2:] = -1
        if t % 4 == 2:
            idx[t, ::2] = [V, V + 5, 2 ** 31 - 1, -3][t // 4 % 4]
        if t % 8 == 7:
            idx[t] = -1
    return idx, val.astype(np.float32)


def check_distill(P, z, idx, val, labels, tau, tail, dkl, dce, mode, inplace=False):
    T, V = z.shape
    dtype, Z = z.dtype, f64(z)
    ref = HO.distill(Z, idx, val, labels, tau, tail, dkl, dce if labels is not None else None)
    a = (dev(idx, torch.int32), dev(val, F32))
    lab = None if labels is None else dev(labels, torch.int32)
    w = dict(dkl=None if dkl is None else dev(dkl, F32), dce=None if dce is None or labels is None else dev(dce, F32))
    kind = dict(labels=lab, temperature=tau, tail=tail)
    if mode == "step":
        o = P.p24_distill_topk(z, *a, **kind, **w, out={"dlogits": z} if inplace else None)
    else:
        o = P.p24_distill_topk(z, *a, **kind)
        assert "dlogits" not in o
        o["dlogits"] = P.p24_distill_topk_bwd(z, *a, o["stats"], **kind, **w, dlogits=z if inplace else None)
    m = Z.max(1, keepdims=True)
    some = m > -np.inf
    x = np.where(some, (Z - np.where(some, m, 0)) / tau, -np.inf)
    x1 = np.where(some, Z - np.where(some, m, 0), -np.inf)
    s, s1 = np.exp(x).sum(1, keepdims=True), np.exp(x1).sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        p, p1 = np.where(some, np.exp(x) / s, 0), np.where(some, np.exp(x1) / s1, 0)
    fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0)  # noqa: E731
    kb, gb, qsum = np.zeros(T), np.zeros((T, V)), np.zeros((T, 1))
    wk, wc = np.abs(dkl if dkl is not None else np.zeros(T)), np.abs(dce if dce is not None else np.zeros(T))
    for t in range(T):
        cols, q, qr = HO.teacher(idx[t], val[t], V, tau, tail)
        with np.errstate(divide="ignore", invalid="ignore"):
            terms = np.where(q > 0, q * (np.abs(np.log(q)) + fin(np.log(p[t, cols]))), 0)
            lr = ref["stats"][t, 2] - ref["stats"][t, 1] if tail and some[t, 0] else 0.0
            kb[t] = 2 * e_s(V) + 16 * U * terms.sum() + (64 * U * (1 + abs(np.log(qr)) + fin(lr)) if tail and qr > 0 else 0)
        qsum[t] = q.sum() + qr
        gb[t, cols] += wk[t] / tau * 8 * U * q * 4
        if tail and qr > 0 and np.isfinite(lr):
            # p (Q - q_r / p_r): the ratio's own error
            qsum[t] += qr / np.exp(lr) * (1 + 64 * U / qr / e_s(V))
    close(o["kl"], ref["kl"], kb, "kl")
    if labels is not None:
        close(o["ce"], ref["ce"], 2 * e_s(V) + 8 * U * fin(ref["ce"]), "ce")
    close(o["stats"], ref["stats"], (2 * e_s(V) + 8 * U * fin(ref["stats"])) * np.array([0, 1, 1, 1]), "stats")
    bound = grad_bound(V, ref["dlogits"], p, x, wk[:, None] / tau * qsum, dtype, gb)
    bound += wc[:, None] * (p1 * (e_s(V) + 4 * U * fin(x1) + 32 * U) + 4 * U)
    close(o["dlogits"], ref["dlogits"], bound, "dlogits")
    return o, ref


DISTILL = [(1, 3, 2, 0), (8, 9, 9, 1), (5, 4099, 16, 0), (3, 50257, 64, 0), (130, 1001, 8, 7), (2, 65536, 128, 0),
           (300, 600, 33, 4), (9, 40, 64, 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,K,pad", DISTILL)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_distill(P, dtype, T, V, K, pad, tail, mode):
    z, rng = logits(T, V, dtype, T + 3 * V + K, pad=pad)
    idx, val = teacher_list(rng, T, V, K)
    labels = rng.integers(0, V, T)
    labels[::3] = np.where(idx[::3, 0] < V, idx[::3, 0], 0)  # a listed label, or an absent one
    labels[1::5] = -100
    dkl, dce = (f64(dev(rng.random(T) + 0.1, F32)) for _ in range(2))
    dkl[::6] = 0
    tau = [1.0, 2.0, 0.7][(T + V + tail) % 3]
    lab = labels if (T + K + (mode == "bwd")) % 2 else None
    check_distill(P, z, idx, val, lab, tau, tail, dkl, dce, mode, inplace=(V % 2 == 0) ^ tail)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,K,pad", [(2, 300001, 40, 0), (170, 40003, 12, 0), (30, 80000, 24, 5), (400, 1000, 128, 0)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_distill_long_rows_and_many_rows(P, dtype, T, V, K, pad, tail, mode):
    """Rows longer than a cluster's registers, rows split over CTAs, more rows than fit at once."""
    z, rng = logits(T, V, dtype, T + V, pad=pad)
    idx, val = teacher_list(rng, T, V, K)
    labels = rng.integers(0, V, T)
    w = f64(dev(rng.random(T), F32))
    check_distill(P, z, idx, val, labels, [1.0, 1.5][T % 4 == 2], tail, w, w[::-1].copy(), mode, inplace=tail)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,k", [(2, 300001, 100), (400, 40003, 64), (500, 1000, 128), (160, 70000, 7)])
def test_score_long_rows_and_many_rows(P, dtype, T, V, k):
    z, rng = logits(T, V, dtype, T + V)
    check_score(P, z, rng.integers(0, V, T), k, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [60.0, 300.0])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_distill_bucket_far_below_the_list(P, dtype, gap, mode):
    """The list holds all but exp(-gap) of the student: p_r underflows, q_r / p_r would overflow,
    and the bucket's loss and gradient are still finite and right."""
    z, rng = logits(3, 5000, dtype, 33, peak=False)
    idx, val = teacher_list(rng, 3, 5000, 4)
    idx[:] = np.array([7, 100, 2500, 4999])
    z[:, torch.as_tensor(idx[0], device="cuda")] += gap
    w = np.ones(3)
    o, ref = check_distill(P, z, idx, val, None, 1.0, True, w, None, mode)
    assert np.all(np.isfinite(ref["kl"])) and np.abs(ref["dlogits"]).max() > 0.01


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_without_a_list_is_cross_entropy(P, dtype, tau, tail):
    z, rng = logits(7, 2050, dtype, 2)
    labels = rng.integers(0, 2050, 7)
    o, ref = check_distill(P, z, np.zeros((7, 0), dtype=np.int64), np.zeros((7, 0), dtype=np.float32), labels, tau, tail,
                           None, np.ones(7), "step")
    assert not ref["kl"].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_distill_masked_rows(P, dtype, tail, mode):
    """Rows masked whole, masked but for the list (nothing is left for the bucket), and with a
    listed entry masked (infinite divergence, finite gradient)."""
    z, rng = logits(8, 3001, dtype, 12)
    idx, val = teacher_list(rng, 8, 3001, 6)
    idx[:] = np.arange(6) * 11 + np.arange(8)[:, None]
    z[0] = float("-inf")
    keep = torch.as_tensor(idx[1], device="cuda")
    left = z[1, keep].clone()
    z[1] = float("-inf")
    z[1, keep] = left
    z[2, int(idx[2, 3])] = float("-inf")
    z[3, 100:] = torch.finfo(dtype).min
    labels = np.array([5, int(idx[1, 0]), 2, 3, -1, 2000, int(idx[6, 2]), 7])
    ones = np.ones(8)
    o, _ = check_distill(P, z, idx, val, labels, 1.0, tail, ones, ones, mode)
    assert not o["dlogits"][0].any() and o["kl"][0].item() == float("inf")


def test_distill_nan(P):
    """A NaN logit or teacher value reaches that row's loss and gradient, and no other row."""
    z, rng = logits(4, 500, F32, 13)
    idx, val = teacher_list(rng, 4, 500, 8)
    idx[:] = np.arange(8)
    z[1, 400] = float("nan")
    val[2, 3] = np.nan
    for tail in (False, True):
        o = P.p24_distill_topk(z, dev(idx, torch.int32), dev(val, F32), tail=tail, dkl=dev(np.ones(4), F32))
        bad = torch.isnan(o["kl"]).tolist()
        assert bad == [False, True, True, False]
        assert torch.isnan(o["dlogits"][1]).all() and torch.isnan(o["dlogits"][2, 3])
        assert not torch.isnan(o["dlogits"][[0, 3]]).any()


def test_gradients_against_differences(P):
    """The fp32 gradients along random directions against central differences of the fp64
    loss: a step of 1e-4 leaves an error of order 1e-8 of the third derivative."""
    z, rng = logits(4, 301, F32, 21)
    idx, val = teacher_list(rng, 4, 301, 12)
    labels = np.array([4, 300, -1, int(idx[3, 0])])
    w, c = rng.random(4), rng.random(4)
    Z, step = f64(z), 1e-4

    def slope(f):
        d = rng.normal(size=Z.shape)
        return d, (f(Z + step * d) - f(Z - step * d)) / (2 * step)

    for tau, tail in ((1.0, False), (2.0, False), (0.7, True)):
        o = P.p24_distill_topk(z, dev(idx, torch.int32), dev(val, F32), dev(labels, torch.int32), temperature=tau,
                               tail=tail, dkl=dev(w, F32), dce=dev(c, F32))
        for _ in range(4):
            d, want = slope(lambda A: sum(b @ r for b, r in zip((w, c), map(
                HO.distill(A, idx, val, labels, tau, tail).get, ("kl", "ce")))))
            assert abs((f64(o["dlogits"]) * d).sum() - want) < 1e-5 * (1 + np.abs(d).max()), (tau, tail)
        s = P.p24_token_logprobs(z, dev(labels, torch.int32), temperature=tau)
        D = P.p24_token_logprobs_bwd(z, dev(labels, torch.int32), s["stats"], dev(w, F32), entropy=s["entropy"],
                                     dentropy=dev(c, F32), temperature=tau)
        d, want = slope(lambda A: sum(b @ r for b, r in zip((w, c), map(
            HO.token_logprobs(A, labels, 0, tau).get, ("logp", "entropy")))))
        assert abs((f64(D) * d).sum() - want) < 1e-5 * (1 + np.abs(d).max()), tau


def test_results_repeat_bit_for_bit_and_on_another_stream(P):
    z, rng = logits(37, 10007, BF, 30)
    idx, val = teacher_list(rng, 37, 10007, 40)
    tok = dev(rng.integers(0, 10007, 37), torch.int32)
    a = (z, dev(idx, torch.int32), dev(val, F32), tok)
    w = dict(tail=True, dkl=dev(rng.random(37), F32), dce=dev(rng.random(37), F32))
    one, two = P.p24_distill_topk(*a, **w), P.p24_token_logprobs(z, tok, k=40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        again, more = P.p24_distill_topk(*a, **w, stream=stream), P.p24_token_logprobs(z, tok, k=40, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(one[n], again[n]) for n in one) and all(torch.equal(two[n], more[n]) for n in two)


def test_row_offsets_past_32_bits(P):
    """Rows whose element offsets pass 2^31 (a wide row stride): the last row is the first."""
    V, T = 1000, 5
    ld = 2 ** 30
    big = torch.empty((T - 1) * ld + V, dtype=BF, device="cuda").as_strided((T, V), (ld, 1))
    z, rng = logits(1, V, BF, 40)
    big[:] = z
    tok = dev(np.full(T, 123), torch.int32)
    o = P.p24_token_logprobs(big, tok, k=7)
    ref = P.p24_token_logprobs(z.expand(T, V).contiguous(), tok, k=7)
    assert all(torch.equal(o[n], ref[n]) for n in ref)
    idx, val = teacher_list(rng, T, V, 9)
    idx[:] = idx[0]
    a = (dev(idx, torch.int32), dev(np.tile(val[:1], (T, 1)), F32))
    w = dict(dkl=dev(np.ones(T), F32), tail=True)
    D = P.p24_distill_topk(big, *a, **w, out={"dlogits": big})["dlogits"]
    want = P.p24_distill_topk(z.expand(T, V).contiguous(), *a, **w)["dlogits"]
    assert torch.equal(D, want)


def test_refusals(P):
    z, _ = logits(3, 100, BF, 50)
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    stats = torch.zeros((3, 2), device="cuda")
    idx, val = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    before = P.p24_launch_count()
    with pytest.raises(TypeError):
        P.p24_token_logprobs(z.half(), tok)
    with pytest.raises(TypeError):
        P.p24_token_logprobs(z, tok.long())
    with pytest.raises(ValueError):
        P.p24_token_logprobs(z.t(), tok)
    with pytest.raises(ValueError):
        P.p24_token_logprobs(z.cpu(), tok)
    with pytest.raises(ValueError):
        P.p24_token_logprobs(z, tok[:2])
    with pytest.raises(ValueError):
        P.p24_token_logprobs(z, tok, out={"logp": torch.empty(4, device="cuda")})
    with pytest.raises(P.P24Error):
        P.p24_token_logprobs(z, tok, k=P.P24_TOPK_MAX + 1)
    with pytest.raises(P.P24Error):
        P.p24_token_logprobs(z, tok, temperature=0.0)
    with pytest.raises(ValueError):
        P.p24_token_logprobs_bwd(z, tok, stats, stats[:, 0].contiguous(), dlogits=z.float())
    with pytest.raises(P.P24Error):
        P.p24_token_logprobs_bwd(z, None, stats, stats[:, 0].contiguous())
    with pytest.raises(ValueError):
        P.p24_distill_topk(z, idx[0], val[0])
    with pytest.raises(TypeError):
        P.p24_distill_topk(z, idx.float(), val)
    with pytest.raises(ValueError):
        P.p24_distill_topk(z, idx, val[:2])
    with pytest.raises(P.P24Error):
        P.p24_distill_topk(z, idx, val, dce=stats[:, 0].contiguous())  # weights of labels that are not given
    assert P.p24_launch_count() == before
    empty = P.p24_token_logprobs(z[:0], tok[:0], k=2)
    assert empty["top_idx"].shape == (0, 2) and P.p24_launch_count() == before
