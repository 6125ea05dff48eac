"""Pins of the oracle of the operators around the sparse FFN (oracle/block_oracle.py): its gradients against
differences, its roundings against enumeration and torch's, its tables against hand-worked cases."""
import numpy as np
import torch

from oracle import block_oracle as BO


def test_rmsnorm_by_hand():
    h, rstd, y = BO.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), eps=0.5)
    assert np.allclose(rstd, 1 / np.sqrt(13.0)) and np.allclose(y, [[3 / np.sqrt(13), 8 / np.sqrt(13)]])
    h, _, _ = BO.rmsnorm(np.array([[1.0, 1.0]]), r=np.array([[2.0 ** -8, 3 * 2.0 ** -8]]), rounded=BO.round_bf16)
    assert np.array_equal(h, [[1.0, 1 + 2 * 2.0 ** -7]])   # both are ties: to the even neighbour


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, dy, dres, w = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    eps = 0.03

    def loss(x, w):
        return (BO.rmsnorm(x, w, eps=eps)[2] * dy).sum() + (x * dres).sum()

    dx, dw = BO.rmsnorm_bwd(dy, x, w, eps, dres)
    s = 1e-5
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = s
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * s) - dx[i, j]) < 1e-8
    for j in range(7):
        e = np.zeros(7)
        e[j] = s
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * s) - dw[j]) < 1e-8


def test_embedding_gradient_is_the_adjoint():
    """<embed(tokens, W), dY> = <W, embed_bwd(dY)> for any W: the lookup is linear."""
    rng = np.random.default_rng(1)
    tokens = np.array([3, 0, 3, -1, 9, 5, 3])     # 5 entries: 9 and 5 are outside
    dY, W = rng.normal(size=(7, 4)), rng.normal(size=(5, 4))
    Y = BO.embed(tokens, W, 1.7)
    assert (Y[[3, 4, 5]] == 0).all()
    assert abs((Y * dY).sum() - (W * BO.embed_bwd(dY, tokens, 5, 1.7)).sum()) < 1e-12
    assert np.allclose(BO.embed_bwd(dY, tokens, 5)[3], dY[0] + dY[2] + dY[6])
    old = rng.normal(size=(5, 4))
    assert np.allclose(BO.embed_bwd(dY, tokens, 5, 2.0, old) - old, BO.embed_bwd(dY, tokens, 5, 2.0))


def test_clip_by_hand():
    n, (a, b) = BO.clip([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert n == 5 and np.allclose(a, [0.6]) and np.allclose(b, [0, 0.8])
    n, (a,) = BO.clip([np.array([0.3])], 1.0)
    assert a[0] == 0.3
    n, (a,) = BO.clip([np.array([np.inf, 2.0])], 1.0)
    assert n == np.inf and a[1] == 2.0


def test_rounding_to_8_bits():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mine = np.array([BO.e4m3_value(c) for c in range(256)])
    assert np.array_equal(codes, mine, equal_nan=True)
    rng = np.random.default_rng(2)
    v = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000), (mine[:126] + mine[1:127]) / 2, mine[:127]])
    v = v.astype(np.float32).astype(np.float64)
    v = v[np.abs(v) <= 448]
    want = torch.as_tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(BO.round_e4m3(v), want)
    assert BO.round_e4m3(1e9) == 448 and BO.round_e4m3(-1e9) == -448


def test_rounding_to_bf16():
    rng = np.random.default_rng(3)
    v = (rng.normal(size=4000) * 10.0 ** rng.integers(-45, 38, 4000)).astype(np.float32).astype(np.float64)
    v = np.concatenate([v, [0.0, np.inf, -np.inf, 3.4e38, 1.0 + 2.0 ** -8, 2.0 ** -133, 3 * 2.0 ** -134]])
    assert np.array_equal(BO.round_bf16(v), torch.as_tensor(v).to(torch.float32).to(torch.bfloat16).double().numpy())


def test_scales():
    y = np.array([[1.0, -448.0, 0, 0, 2.0]])
    assert np.array_equal(BO.scales(y, 0), [[1.0]])
    assert np.allclose(BO.scales(y, 2), [[1.0, 1.0, 2 / 448]])   # a group of zeros has 1
    assert np.array_equal(BO.spread(np.array([[1.0, 2.0, 3.0]]), 5, 2), [[1, 1, 2, 2, 3]])


def test_a_planted_mistake_is_caught():
    """The gradient without the projection along xh fails the differences."""
    x, dy = np.array([[1.0, 2.0, -1.0]]), np.array([[0.5, 0.1, 0.3]])
    dx, _ = BO.rmsnorm_bwd(dy, x, None, 1e-6)
    assert abs((dx * x).sum()) < 1e-6              # along x the norm does not change
    wrong = dy / np.sqrt((x * x).mean())
    assert abs((wrong * x).sum()) > 0.1
