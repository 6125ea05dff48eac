"""Pins of the head operators' oracle (oracle/head_oracle.py), on the CPU: closed forms,
a brute-force ordering, its gradients against central differences in fp64, and against the
other formulations the definitions reduce to."""
import numpy as np
import pytest

from oracle import head_oracle as HO


def rng_logits(T, V, seed, sigma=2.0):
    return np.random.default_rng(seed).normal(size=(T, V)) * sigma


def test_uniform_and_two_point_rows_in_closed_form():
    Z = np.array([[3.0, 3.0, 3.0, 3.0], [np.log(3.0), 0.0, -np.inf, -np.inf]])
    o = HO.token_logprobs(Z, np.array([2, 1]), k=4)
    assert np.allclose(o["logp"], [-np.log(4), -np.log(4)])
    assert np.allclose(o["entropy"], [np.log(4), 0.25 * np.log(4) + 0.75 * np.log(4 / 3)])
    assert o["top_idx"].tolist() == [[0, 1, 2, 3], [0, 1, 2, 3]]
    assert np.allclose(o["top_logp"][1, :2], np.log([0.75, 0.25])) and np.all(o["top_logp"][1, 2:] == -np.inf)


def test_order_of_special_values():
    z = np.array([0.0, -0.0, np.inf, np.nan, -np.inf, 1.0, np.nan])
    assert HO.order(z).tolist() == [3, 6, 2, 5, 0, 1, 4]


def test_empty_row_and_absent_tokens():
    Z = np.full((2, 5), -np.inf)
    Z[1] = 0.0
    o = HO.token_logprobs(Z, np.array([1, -1]), k=2)
    assert o["logp"][0] == -np.inf and o["logp"][1] == 0 and o["entropy"][0] == 0
    assert not HO.token_logprobs_bwd(Z, np.array([1, -1]), np.ones(2), None).any()


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.0])
def test_logprob_gradient_against_differences(tau):
    Z = rng_logits(3, 17, 5)
    Z[1, 4] = -np.inf
    tokens, g, h = np.array([3, 9, 40]), np.array([0.7, -1.1, 2.0]), np.array([0.3, 0.2, -0.5])

    def loss(A):
        o = HO.token_logprobs(A, tokens, tau=tau)
        return (g * o["logp"]).sum() + (h * o["entropy"]).sum()

    D = HO.token_logprobs_bwd(Z, tokens, g, h, tau)
    check_differences(loss, Z, D)


def check_differences(loss, Z, D, step=1e-5):
    for t in range(Z.shape[0]):
        for j in range(Z.shape[1]):
            if Z[t, j] == -np.inf:
                assert D[t, j] == 0
                continue
            up, dn = Z.copy(), Z.copy()
            up[t, j] += step
            dn[t, j] -= step
            assert abs((loss(up) - loss(dn)) / (2 * step) - D[t, j]) < 1e-8, (t, j)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distillation_gradient_against_differences(tail, tau):
    Z = rng_logits(4, 19, 7)
    rng = np.random.default_rng(8)
    idx = np.stack([rng.permutation(19)[:5] for _ in range(4)])
    idx[1, 2] = -1
    idx[2, :] = 30
    val = np.log(rng.dirichlet(np.ones(6), size=4)[:, :5])
    labels = np.array([idx[0, 0], 3, 18, -1])
    dkl, dce = np.array([1.0, 0.5, 2.0, 0.1]), np.array([0.3, 0.0, 1.0, 5.0])

    def loss(A):
        o = HO.distill(A, idx, val, labels, tau, tail)
        return (dkl * o["kl"]).sum() + (dce * o["ce"]).sum()

    o = HO.distill(Z, idx, val, labels, tau, tail, dkl, dce)
    check_differences(loss, Z, o["dlogits"])


def test_a_list_of_the_whole_vocabulary_is_the_plain_divergence():
    """K = V: both forms are KL(teacher || student), 0 for the teacher itself."""
    Z = rng_logits(2, 6, 1)
    lp = Z - np.log(np.exp(Z).sum(1, keepdims=True))
    S = rng_logits(2, 6, 2)
    ls = S - np.log(np.exp(S).sum(1, keepdims=True))
    idx = np.tile(np.arange(6), (2, 1))
    want = (np.exp(lp) * (lp - ls)).sum(1)
    for tail in (False, True):
        assert np.allclose(HO.distill(S, idx, lp, tail=tail)["kl"], want)
        assert np.allclose(HO.distill(Z, idx, lp, tail=tail)["kl"], 0)


def test_tail_divergence_is_that_of_the_merged_vocabulary():
    """The bucket form equals KL over K + 1 outcomes with the rest merged into one."""
    Z, S = rng_logits(1, 9, 3), rng_logits(1, 9, 4)
    p = np.exp(Z[0]) / np.exp(Z[0]).sum()
    s = np.exp(S[0]) / np.exp(S[0]).sum()
    cols = np.array([7, 0, 4])
    merged = lambda a: np.append(a[cols], np.delete(a, cols).sum())  # noqa: E731
    want = (merged(p) * np.log(merged(p) / merged(s))).sum()
    got = HO.distill(S, cols[None], np.log(p[cols])[None], tail=True)["kl"][0]
    assert np.isclose(got, want)


def test_planted_mistake_in_the_tail_gradient_is_caught():
    """Dropping the bucket's term from the unlisted columns breaks the difference check."""
    Z = rng_logits(1, 9, 5)
    idx, val = np.array([[1, 2]]), np.log(np.array([[0.4, 0.3]]))
    o = HO.distill(Z, idx, val, tail=True, dkl=np.ones(1))
    p = np.exp(Z) / np.exp(Z).sum()
    wrong = p.copy()
    wrong[0, idx[0]] -= np.exp(val[0])
    assert np.abs(o["dlogits"] - wrong).max() > 1e-2
    with pytest.raises(AssertionError):
        check_differences(lambda A: HO.distill(A, idx, val, tail=True)["kl"].sum(), Z, wrong)
