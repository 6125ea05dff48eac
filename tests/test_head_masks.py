"""Rows of logits masked by a finite value: alternatives where fewer entries are left than asked
for, and the bucket of the rest where everything in it is masked. Helpers and tolerances are those
of test_parity_head unless a test derives its own."""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO
from tests.test_parity_head import BF, F32, P, U, close, dev, e_s, f64  # noqa: F401

pytestmark = pytest.mark.gpu

# just above fp32's lowest value, its lowest value, and fp32 copies of a bf16 mask
LOWS = {"3.4e38": -3.4e38, "lowest": torch.finfo(F32).min, "bf16 lowest": torch.finfo(BF).min}


@pytest.mark.parametrize("low", LOWS)
@pytest.mark.parametrize("T,V", [(700, 20011), (8, 300001)])
def test_alternatives_of_fp32_rows_masked_near_the_lowest_value(P, T, V, low):  # noqa: F811
    """0 to k - 1 entries left of a row, at every alignment of a row to 16 bytes and so with 0 to 6
    elements outside its aligned vectors: the masked ones come after the live ones, in order of position."""
    rng = np.random.default_rng(V)
    ld = V + (1 - V) % 4  # row t starts t elements past a 16-byte boundary
    z = torch.empty((T, ld), dtype=F32, device="cuda")[:, :V]
    z.fill_(LOWS[low])
    for t in range(T):
        live = rng.permutation(V)[:t // 4 % 6]
        z[t, torch.as_tensor(live, device="cuda")] = torch.as_tensor(rng.normal(size=len(live)), device="cuda").float()
    want = np.stack([HO.order(r)[:6] for r in f64(z)])
    for k in range(1, 7):
        got = P.p24_token_logprobs(z, k=k)["top_idx"].cpu().numpy()
        bad = np.nonzero((got != want[:, :k]).any(1))[0]
        assert not len(bad), (k, bad[:8], got[bad[0]], want[bad[0], :k])


def bucket(z, idx, val, labels, tau, dkl, dce):
    """One row's kl, and gradient with the softmax of what is off the list taken by itself, in fp64:
    (Q p_r - q_r) softmax(z_off / tau) holds however small p_r is."""
    x = z / tau
    off = np.ones(len(z), dtype=bool)
    off[idx] = False
    lse = lambda a: a.max() + np.log(np.exp(a - a.max()).sum())  # noqa: E731
    ls, lr = lse(x), lse(x[off])
    q = np.exp(val.astype(np.float64))
    qr = 1 - q.sum()
    kl = (q * (np.log(q) - (x[idx] - ls))).sum() + qr * (np.log(qr) - (lr - ls))
    p = np.exp(x - ls)
    g = (q.sum() + qr) * p
    rest = np.exp(x[off] - x[off].max())  # at its own reference: lr takes the last digits even of fp64 with it
    rest /= rest.sum()
    g[off] = ((q.sum() + qr) * np.exp(lr - ls) - qr) * rest
    g[idx] -= q
    p1 = np.exp(z - lse(z))
    d = dkl / tau * g + dce * p1
    d[labels] -= dce
    return kl, d, qr


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mask", [-1e4, -1e9, "lowest"])
@pytest.mark.parametrize("tau", [1.0, 0.5, 2.0])
@pytest.mark.parametrize("T,V", [(3, 5003), (200, 1001), (2, 40001)])
@pytest.mark.parametrize("mode", ["step", "bwd", "inplace"])
def test_bucket_of_masked_logits(P, dtype, mask, tau, T, V, mode):  # noqa: F811
    """Every logit off the list is masked by one finite value or lies near it: the bucket's gradient
    is spread over them as their own softmax says, -q_r in total.

    Tolerance: q_r = 1 - sum q is off by at most 64u, relative 64u / q_r; an element off the list
    by that, by e_s of its sum, and by 8u + 4u |x| of its exponential, x its distance to the largest
    one off the list over tau (at most 8 / 0.5); fp32's smallest normal number absolutely. The terms on the list are bounded as
    in test_parity_head. The loss is q_r times a distance that takes four roundings, so it is off by
    (64u / q_r + 8u) relative, and by the list's own terms."""
    rng = np.random.default_rng(int(V + 10 * tau))
    low = torch.finfo(dtype).min if mask == "lowest" else mask
    K = 8
    idx = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    val = np.log(rng.dirichlet(np.ones(K), size=T) * 0.9 + 1e-3).astype(np.float32)
    z = torch.full((T, V), low, dtype=dtype, device="cuda")
    step = 1.0 if mask == -1e4 else 0.0  # near the mask, not only at it: one apart is representable there in fp32
    if step and dtype == F32:
        z -= step * torch.as_tensor(rng.integers(0, 8, (T, V)), device="cuda").float()
    z.scatter_(1, dev(idx, torch.int64), dev(rng.normal(size=(T, K)) * 2, dtype))
    labels = idx[:, 2]
    w, c = f64(dev(rng.random(T) + 0.1, F32)), f64(dev(rng.random(T), F32))
    Z = f64(z)
    a = (z, dev(idx, torch.int32), dev(val, F32), dev(labels, torch.int32))
    kind, weights = dict(temperature=tau, tail=True), dict(dkl=dev(w, F32), dce=dev(c, F32))
    if mode == "step":
        o = P.p24_distill_topk(*a, **kind, **weights)
    else:
        o = P.p24_distill_topk(*a, **kind)
        o["dlogits"] = P.p24_distill_topk_bwd(*a[:3], o["stats"], labels=a[3], **kind, **weights,
                                              dlogits=z if mode == "inplace" else None)
    for t in range(T):
        kl, d, qr = bucket(Z[t], idx[t], val[t], labels[t], tau, w[t], c[t])
        assert abs(o["kl"][t].item() - kl) <= (64 * U / qr + 8 * U) * abs(kl) + 2 * e_s(V) + 64 * U * (1 + abs(np.log(qr))) * 8
        rel = np.full(V, e_s(V) + 8 * U + 4 * U * 16 + 64 * U / qr)
        rel[idx[t]] = e_s(V) + 256 * U
        bound = rel * np.abs(d) + 2.0 ** -126 + (2.0 ** -8 * np.abs(d) if dtype == BF else 0)
        bound[idx[t]] += (w[t] / tau + c[t]) * (e_s(V) + 64 * U)  # differences of terms of at most the weights
        close(o["dlogits"][t], d, bound, ("dlogits", t))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [False, True])
def test_masked_token_label_and_listed_entry(P, dtype, tail):  # noqa: F811
    """A logit of -inf that the row's token, label or list names: infinite losses, and its delta or q term
    alone as its gradient. Values: one fp32 product or quotient and the output's rounding."""
    V, tau = 1003, 2.0
    z = torch.randn((3, V), device="cuda").to(dtype)
    z[:, 17] = float("-inf")
    tok = dev(np.full(3, 17), torch.int32)
    w, c = dev(np.array([1.5, -0.5, 0.3]), F32), dev(np.array([0.7, 0.2, 1.1]), F32)
    o = P.p24_token_logprobs(z, tok, temperature=tau)
    assert (o["logp"] == float("-inf")).all()
    D = P.p24_token_logprobs_bwd(z, tok, o["stats"], w, temperature=tau)
    rel = 2.0 ** -8 if dtype == BF else 4 * U
    close(D[:, 17], f64(w) / tau, rel * np.abs(f64(w)), "token")
    assert torch.isfinite(D).all()
    idx = dev(np.tile([3, 17], (3, 1)), torch.int32)
    val = torch.log(dev(np.tile([0.5, 0.3], (3, 1)), F32))
    q = 0.3 if tail else np.sqrt(0.3) / (np.sqrt(0.5) + np.sqrt(0.3))
    s = P.p24_distill_topk(z, idx, val, tok, temperature=tau, tail=tail, dkl=w, dce=c)
    assert (s["kl"] == float("inf")).all() and (s["ce"] == float("inf")).all()
    back = P.p24_distill_topk_bwd(z, idx, val, s["stats"], w, tok, c, temperature=tau, tail=tail)
    want = -f64(w) / tau * q - f64(c)
    for d in (s["dlogits"], back):
        close(d[:, 17], want, (rel + 16 * U) * (np.abs(f64(w)) + np.abs(f64(c))), "label and list")
        assert torch.isfinite(d).all()
