"""One meaning of a teacher's list in DistillHead: log probabilities at the temperature in use,
with the bucket and without, as teacher_list gives them."""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO
from synth24 import normal_bf16
from tests.test_parity_head import U, close, e_s, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("with_labels", [False, True])
def test_list_and_step_at_one_temperature(tau, tail, with_labels):
    """kl, ce and the logits' gradient against fp64 from the two models' logits alone: the teacher's
    probabilities are softmax(teacher / tau), on the list renormalised or with the bucket.

    Tolerance: the list's values are off by e_s + 8u |value| + 8u ln s, which is a relative error of
    each q (again 8u for a product and a quotient by the temperature); kl = sum q (ln q - ln p) turns
    it into (1 + |ln q - ln p|) of the same, beside the student's own error; the bucket's q_r by 64u
    and the q's errors. Gradients: q's errors and p's on top of bf16's rounding."""
    import semi_structured_sparse_prune24_gb300 as P
    from semi_structured_sparse_prune24_gb300.distill import DistillHead
    M, d, V, K = 40, 128, 2000, 24
    Yt, Wt = normal_bf16((M, d), 1.0, 7, 1, "cuda"), normal_bf16((V, d), 0.3, 7, 2, "cuda")
    Y, W = normal_bf16((M, d), 1.0, 7, 3, "cuda"), normal_bf16((V, d), 0.3, 7, 4, "cuda")
    head = DistillHead(M, d, V)
    t = head.teacher_list(Yt, Wt, K, temperature=tau)
    Zt = head.logits.double().cpu().numpy()
    labels = (torch.arange(M, dtype=torch.int32, device="cuda") * 37) % V if with_labels else None
    w = torch.linspace(0.5, 1.5, M, device="cuda")
    c = 0.5 * w if with_labels else None
    Z = P.p24_gemm_nt(Y, W).double().cpu().numpy()
    o = head.step(Y, W, t["top_idx"], t["top_logp"], w, labels, c, temperature=tau, tail=tail)
    torch.cuda.synchronize()
    assert P.p24_query_status() == 0
    idx = t["top_idx"].cpu().numpy()
    lse = lambda a: a.max(-1, keepdims=True) + np.log(np.exp(a - a.max(-1, keepdims=True)).sum(-1, keepdims=True))  # noqa: E731
    lq, lp, l1 = Zt / tau - lse(Zt / tau), Z / tau - lse(Z / tau), Z - lse(Z)
    rows = np.arange(M)[:, None]
    assert np.array_equal(idx, np.stack([HO.order(r)[:K] for r in Zt]))
    q = np.exp(lq[rows, idx])
    off = np.ones((M, V), dtype=bool)
    off[rows, idx] = False
    p = np.exp(lp)
    e_q = e_s(V) + 8 * U * (np.abs(lq[rows, idx]).max() + 10) + 32 * U   # relative, of each q
    xs = np.abs(Z - Z.max(1, keepdims=True))
    e_p = e_s(V) + 4 * U * xs / tau + 128 * U                            # relative, of each p
    if tail:
        qr = 1 - q.sum(1)
        pr = np.where(off, p, 0).sum(1)
        kl = (q * (np.log(q) - lp[rows, idx])).sum(1) + qr * (np.log(qr) - np.log(pr))
        g = np.where(off, p * (1 - qr / pr)[:, None], p)
        e_r = 64 * U + 2 * e_q                       # absolute, of q_r
        far = np.abs(np.log(qr) - np.log(pr)) + 1
        spread = np.where(off, p / pr[:, None], 0)
    else:
        q = q / q.sum(1, keepdims=True)
        kl = (q * (np.log(q) - lp[rows, idx])).sum(1)
        g, e_r, far, spread = p.copy(), 0.0, 1.0, 0.0
    g[rows, idx] -= q
    terms = (q * (1 + np.abs(np.log(q) - lp[rows, idx]))).sum(1)
    close(o["kl"], kl, 2 * e_q * terms + 4 * e_s(V) + e_r * far, "kl")
    D = f64(w)[:, None] / tau * g
    if with_labels:
        lab = labels.cpu().numpy()
        close(o["ce"], -l1[np.arange(M), lab], 2 * e_s(V) + 8 * U * np.abs(l1).max(), "ce")
        D += f64(c)[:, None] * np.exp(l1)
        D[np.arange(M), lab] -= f64(c)
    total = f64(w)[:, None] / tau
    bound = 2.0 ** -8 * np.abs(D) + total * (p * e_p + spread * (2 * e_r + e_p)) + 1e-38
    np.add.at(bound, (rows, idx), total * q * 2 * e_q)
    if with_labels:
        bound += f64(c)[:, None] * (np.exp(l1) * (e_s(V) + 4 * U * xs + 128 * U) + 4 * U)
    close(head.logits, D, bound, "dlogits")
