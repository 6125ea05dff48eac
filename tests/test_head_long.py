"""The head's row operators at the longest rows they take: V = 2^30 (2^19 with the bucket), and rows of
odd length beyond 2^28 fp32 elements at odd alignments. References in fp64 on the device, by chunks."""
import numpy as np
import pytest
import torch

from tests.test_parity_head import BF, F32, P, U, check_distill, e_s, f64, logits, teacher_list  # noqa: F401

pytestmark = pytest.mark.gpu
CHUNK = 1 << 27


def chunks(V):
    return [slice(i, min(V, i + CHUNK)) for i in range(0, V, CHUNK)]


def rows(T, V, dtype, pad):
    z = torch.empty((T, V + pad), dtype=dtype, device="cuda")[:, :V]
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    for t in range(T):
        for c in chunks(V):
            z[t, c] = torch.randn(c.stop - c.start, generator=g, device="cuda") * 2.5
    return z


def order_of_best(row, k):
    """The k best columns, ties to the lower one: from those that reach the k-th value of all chunks."""
    least = torch.cat([row[c].topk(min(k, c.stop - c.start)).values for c in chunks(len(row))]).topk(k).values[-1]
    at = torch.cat([(row[c] >= least).nonzero()[:, 0] + c.start for c in chunks(len(row))])
    return at[row[at].sort(descending=True, stable=True).indices][:k]


@pytest.mark.parametrize("T,V,dtype,pad", [(2, 1 << 30, BF, 0), (3, (1 << 28) + 3, F32, 2)])
def test_longest_rows(P, T, V, dtype, pad):  # noqa: F811
    """Log probabilities, entropy, alternatives, both gradients in place. Tolerances as in test_parity_head:
    e_s(V) of the sums, which is V / 512 roundings of one thread's additions."""
    z = rows(T, V, dtype, pad)
    tokens = torch.tensor([V - 1, 5, V // 2 + 1][:T], dtype=torch.int32, device="cuda")
    o = P.p24_token_logprobs(z, tokens, k=64)
    e, spot = e_s(V), [0, 1, 7, V // 3, V - 2, V - 1]
    ref = []
    for t in range(T):
        assert torch.equal(o["top_idx"][t].long(), order_of_best(z[t], 64)), t
        m = z[t].max().double().item()
        s = sum((z[t, c].double() - m).exp().sum().item() for c in chunks(V))
        a = sum(((z[t, c].double() - m).exp() * (z[t, c].double() - m)).sum().item() for c in chunks(V))
        ls = np.log(s)
        x = z[t, tokens[t].long()].double().item() - m
        assert abs(o["stats"][t, 1].item() - ls) <= e + 8 * U * ls
        assert abs(o["logp"][t].item() - (x - ls)) <= e + 8 * U * (ls + abs(x - ls))
        assert abs(o["entropy"][t].item() - (ls - a / s)) <= (e + 8 * U * ls) * (2 + np.log(V))
        ref.append((m, ls, z[t, spot].double().cpu().numpy()))
    idx = torch.tensor([[V - 1, 3, V // 2, V - 70000]] * T, dtype=torch.int32, device="cuda")
    val = torch.log(torch.tensor([[0.4, 0.3, 0.2, 0.1]] * T, device="cuda"))
    w = torch.ones(T, device="cuda")
    listed = z[:, idx[0].long()].double()
    d = P.p24_distill_topk(z, idx, val, dkl=w)
    for t in range(T):
        m, ls, x = ref[t]
        p = np.exp(x - m - ls)
        want = p - np.array([0, 0, 0, 0, 0, 0.4])
        bound = p * 2 * e + 0.4 * 16 * U + 2.0 ** -8 * np.abs(want)
        assert (np.abs(f64(d["dlogits"][t, spot]) - want) <= bound).all(), t
        q = torch.tensor([0.4, 0.3, 0.2, 0.1], dtype=torch.float64, device="cuda")
        kl = (q * (q.log() - (listed[t] - m - ls))).sum().item()
        assert abs(d["kl"][t].item() - kl) <= 2 * e + 64 * U * 30
    total = d["dlogits"]
    for t in range(T):  # what is off the list is p: the sum is that of the probabilities, less q
        got = sum(total[t, c].double().sum().item() for c in chunks(V))
        assert abs(got) <= 2 * e + 2.0 ** -8
    del d, total
    P.p24_token_logprobs_bwd(z, tokens, o["stats"], w, dlogits=z)
    for t in range(T):
        m, ls, x = ref[t]
        want = -np.exp(x - m - ls)
        want += np.array([tokens[t].item() == (i % V) for i in spot])
        bound = np.exp(x - m - ls) * 2 * e + 2.0 ** -8 * np.abs(want) + 4 * U
        assert (np.abs(f64(z[t, spot]) - want) <= bound).all(), t


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_longest_rows_with_the_bucket(P, dtype, mode):  # noqa: F811
    T, V = 3, 1 << 19
    z, rng = logits(T, V, dtype, 77)
    idx, val = teacher_list(rng, T, V, 128)
    idx[0, :4] = [0, V - 1, V - 2, 1]
    w = np.ones(T)
    check_distill(P, z, idx, val, rng.integers(0, V, T), 1.0, True, w, w, mode)
