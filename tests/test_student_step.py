"""StudentStep: tokens to clipped gradients, against autograd in fp64 on the GPU.

The weights are 2:4 along both axes ((row + column) % 4 < 2 is kept), so that the prune and the double prune keep exactly
what is there, and the gradient through the double-pruned products is the true one. Then every difference is
rounding: 14 bf16 roundings at most lie on the way from the inputs to a gradient (embedding, norm, H, Y, h, norm,
logits' gradient, dY, dh, dH, dn, dx, the weight's gradient, and clipping), each off by at most 2^-8 of the value;
sums of products of random sign keep that ratio of the norms. Normwise bound: 14 * 2^-8 = 5.5e-2; for the
losses, that of the logits (6 roundings) times their norm per token."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def both_ways(rows, cols, g, sigma):
    w = torch.randn((rows, cols), generator=g, device="cuda") * sigma
    w = torch.where(w.abs() < 0.05 * sigma, 0.05 * sigma, w)      # nothing that is kept is zero
    keep = (torch.arange(rows, device="cuda")[:, None] + torch.arange(cols, device="cuda")) % 4 < 2
    return (w * keep).to(BF), keep


def inputs(M, d, ffn, V, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W_up, k_up = both_ways(ffn, d, g, 0.1)
    W_down, k_down = both_ways(d, ffn, g, 0.1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = dict(E=(rnd(V, d) * 0.5).to(BF), w_in=1 + 0.1 * rnd(d), W_up=W_up, b_up=0.1 * rnd(ffn), W_down=W_down,
             b_down=0.1 * rnd(d), w_out=1 + 0.1 * rnd(d), W_head=(rnd(V, d) * 0.1).to(BF))
    tokens = (torch.rand(M, generator=g, device="cuda") ** 3 * V).to(torch.int32)
    tokens[::9] = -1
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(M)]).to(torch.int32)
    val = torch.log_softmax(rnd(M, K), 1) + np.log(0.8)
    return w, dict(up=k_up, down=k_down), tokens, idx, val


def exact(w, keep, tokens, idx, val, dkl, scale, eps, tied):
    """The loss sum(dkl kl), with a bucket, and its gradients."""
    leaf = {k: v.double().requires_grad_(True) for k, v in w.items() if not (tied and k == "W_head")}
    E, head = leaf["E"], leaf["E"] if tied else leaf["W_head"]
    ok = (tokens >= 0).double()[:, None]
    x = E[tokens.clamp_min(0).long()] * scale * ok

    def norm(a, weight):
        return a / torch.sqrt(a.square().mean(1, keepdim=True) + eps) * weight
    H = torch.relu(norm(x, leaf["w_in"]) @ leaf["W_up"].T + leaf["b_up"])
    h = x + H @ leaf["W_down"].T + leaf["b_down"]
    lp = torch.log_softmax(norm(h, leaf["w_out"]) @ head.T, 1)
    q, at = val.double().exp(), idx.long()
    qr = 1 - q.sum(1)
    pr = 1 - lp.gather(1, at).exp().sum(1)
    kl = (q * (q.log() - lp.gather(1, at))).sum(1) + qr * (qr.log() - pr.log())
    grads = torch.autograd.grad((kl * dkl.double()).sum(), list(leaf.values()))
    out = {"d" + k: g for k, g in zip(leaf, grads)}
    out["dW_up"], out["dW_down"] = out["dW_up"] * keep["up"], out["dW_down"] * keep["down"]
    return kl.detach(), out


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("M,d,ffn,V", [(256, 128, 256, 512), (200, 264, 520, 1000)])
def test_step(P, tied, M, d, ffn, V):
    from semi_structured_sparse_prune24_gb300.distill import StudentStep
    w, keep, tokens, idx, val = inputs(M, d, ffn, V, 8, M + tied)
    if tied:
        w["W_head"] = None
    dkl = torch.full((M,), 3.0 / M, device="cuda")
    step = StudentStep(M, d, ffn, V, scale=1.5, eps=1e-5)
    o = step.run(tokens, w, idx, val, dkl, max_norm=None)
    kl, want = exact({k: v for k, v in w.items() if v is not None}, keep, tokens, idx, val, dkl, 1.5, 1e-5, tied)
    assert float((o["kl"].double() - kl).norm() / kl.norm()) <= 6 * 2 ** -8
    assert set(step.gradients(tied)) == set(want)
    for k in want:
        rel = float((o[k].double() - want[k]).norm() / want[k].norm())
        assert rel <= 14 * 2 ** -8, (k, rel)
    # the same step clipped: every gradient scaled by one factor, and the norm they had
    c = step.run(tokens, w, idx, val, dkl, max_norm=1e-2)
    n = float(torch.stack([o[k].double().square().sum() for k in want]).sum().sqrt())
    assert abs(float(c["norm"]) - n) <= 1e-6 * n and n > 1e-2
    for k in want:
        a, b = c[k].double(), o[k].double() * 1e-2 / n
        assert bool(((a - b).abs() <= (torch.finfo(c[k].dtype).eps / 2 + 1e-6) * b.abs() + 2.0 ** -134).all()), k


def test_step_on_another_stream_and_in_a_graph(P):
    """The same numbers on another stream, and from a captured step replayed on new inputs. db_up is summed by atomics,
    whose order is free: it and what is scaled by a norm that has it in are left out, or compared to rounding."""
    from semi_structured_sparse_prune24_gb300.distill import StudentStep
    M, d, ffn, V = 256, 128, 256, 512
    w, _, tokens, idx, val = inputs(M, d, ffn, V, 8, 1)
    w2, _, tokens2, idx2, val2 = inputs(M, d, ffn, V, 8, 2)
    dkl = torch.full((M,), 1.0 / M, device="cuda")
    step = StudentStep(M, d, ffn, V)
    names = [k for k in step.gradients() if k != "db_up"] + ["kl"]
    eager = [step.run(*a, dkl, max_norm=None) for a in ((tokens, w, idx, val), (tokens2, w2, idx2, val2))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step.run(tokens, w, idx, val, dkl, max_norm=None, stream=s)
    s.synchronize()
    assert all(torch.equal(got[k], eager[0][k]) for k in names)
    buf = [tokens.clone(), {k: v.clone() for k, v in w.items()}, idx.clone(), val.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step.run(buf[0], buf[1], buf[2], buf[3], dkl, max_norm=0.25)
    for k, (t, ww, i, v) in enumerate(((tokens, w, idx, val), (tokens2, w2, idx2, val2), (tokens, w, idx, val))):
        buf[0].copy_(t), buf[2].copy_(i), buf[3].copy_(v)
        for n in ww:
            buf[1][n].copy_(ww[n])
        g.replay()
        torch.cuda.synchronize()
        ref = eager[k % 2]
        assert torch.equal(out["kl"], ref["kl"])
        n = float(torch.stack([ref[x].double().square().sum() for x in step.gradients()]).sum().sqrt())
        assert abs(float(out["norm"]) - n) <= 1e-6 * n
        for x in names[:-1]:
            b = ref[x].double() * min(1.0, 0.25 / n)
            assert bool(((out[x].double() - b).abs() <= (torch.finfo(ref[x].dtype).eps / 2 + 2e-6) * b.abs() + 2.0 ** -134).all()), x


def test_a_step_is_refused_inputs_of_other_sizes(P):
    from semi_structured_sparse_prune24_gb300.distill import StudentStep
    w, _, tokens, idx, val = inputs(64, 64, 64, 64, 4, 3)
    step = StudentStep(64, 64, 64, 64)
    dkl = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        step.run(tokens[:32], w, idx, val, dkl)
    for k in ("E", "w_in", "W_up", "W_head"):
        with pytest.raises(ValueError):
            step.run(tokens, {**w, k: w[k][:32]}, idx, val, dkl)


@pytest.mark.parametrize("absent", [("b_up", "b_down"), ("w_in", "w_out"), ("w_out", "b_up")])
def test_a_step_without_some_norms_or_biases(P, absent):
    """They have no gradient, the norm counts none for them, and the others are those of ones and zeros in their place."""
    from semi_structured_sparse_prune24_gb300.distill import StudentStep
    w, _, tokens, idx, val = inputs(64, 64, 64, 64, 4, 3)
    dkl = torch.full((64,), 1.0 / 64, device="cuda")
    step = StudentStep(64, 64, 64, 64)
    o = step.run(tokens, {k: v for k, v in w.items() if k not in absent}, idx, val, dkl, max_norm=1e9)
    neutral = {k: (v if k not in absent else torch.ones_like(v) if k[0] == "w" else torch.zeros_like(v)) for k, v in w.items()}
    want = step.run(tokens, neutral, idx, val, dkl, max_norm=None)
    names = [k for k in step.gradients() if k[1:] not in absent]
    assert set(names) | {"kl", "norm"} <= set(o) and not any("d" + k in o for k in absent)
    for k in names:
        if k != "db_up":        # by atomics
            assert torch.equal(o[k], want[k]), k
    n = float(torch.stack([o[k].double().square().sum() for k in names]).sum().sqrt())
    assert abs(float(o["norm"]) - n) <= 1e-6 * n
    for k in ("E", "W_up", "W_down"):
        with pytest.raises(ValueError, match=k):
            step.run(tokens, {**w, k: None}, idx, val, dkl)
