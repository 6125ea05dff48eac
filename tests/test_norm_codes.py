"""The 8-bit codes of p24_rmsnorm, one by one: a code is the value / scale, both as the call holds them, divided in fp32 and
rounded to nearest even.

The values follow from the call's own h and rstd: h rstd and its product with the weight are each rounded to fp32 once, as
numpy does here, so codes and a group's scale, the largest magnitude times fp32's 1 / 448, have to be equal. A row's scale
comes from the largest |h w| times rstd: two roundings of products on either way, and the last product's on both, 6 steps of 2^-24.
The rows are integers up to 448 with weights of few bits: many quotients lie on the midpoint of two codes or a step of fp32
beside it, where every other way to divide shows."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def check(P, x, w, r, group, rows_of=None):
    T, d = x.shape
    buf = torch.zeros(T * d if rows_of is None else T * rows_of, dtype=torch.uint8, device="cuda")
    y8 = buf.view(T, -1)[:, :d].view(E4) if rows_of is None else buf.view(E4).view(T, rows_of)[:, :d]
    o = P.p24_rmsnorm(x, w, residual=r, group=group, out={"y": y8})
    h = (x if r is None else o["h"]).float().cpu().numpy()
    n = group or d
    with np.errstate(over="ignore", invalid="ignore"):
        y = (h * o["rstd"].cpu().numpy()[:, None]) * w.float().cpu().numpy()
        assert y.dtype == np.float32
        top = np.stack([np.abs(y[:, c:c + n]).max(1) for c in range(0, d, n)], 1)
        want = np.where(top == 0, np.float32(1), np.maximum(top * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -118)))
        scale = o["scale"].cpu().numpy()
        if group and group < d:
            assert np.array_equal(scale, want)
        else:
            fin = np.isfinite(want)
            assert np.array_equal(np.isfinite(scale), fin)
            assert (np.abs(scale.astype(np.float64) - want) <= 6 * U * want)[fin].all()
        q = y / BO.spread(scale, d, n)
    assert q.dtype == np.float32
    code, got = BO.round_e4m3(q), o["y"].float().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(code))
    off = (got != code) & ~np.isnan(code)
    assert not off.any(), (int(off.sum()), off.size, q[off][:4], got[off][:4], code[off][:4])
    assert np.array_equal(np.signbit(got), np.signbit(q) & ~np.isnan(q)) or np.isnan(q).any()
    return o


def integers(T, d, seed, pad=0, dtype=BF):
    rng = np.random.default_rng(seed)
    a = rng.integers(-56, 57, (T, d)) * 8.0 / 2.0 ** rng.integers(0, 5, (T, d))
    a[:, rng.integers(0, d, 1 + d // 40)] = 448.0
    v = torch.zeros((T, d + pad), dtype=dtype, device="cuda")[:, :d]
    v.copy_(torch.as_tensor(a, device="cuda"))
    w = torch.as_tensor(rng.choice([1.0, 0.5, 1.25, -1.5, 0.875, 1.0625], d), device="cuda")
    return v, w


@pytest.mark.parametrize("T,d", [(5, 40), (700, 130), (300, 512), (400, 768), (64, 1024), (700, 2056), (3, 4096), (700, 4096), (40, 8192), (3, 20000)])
@pytest.mark.parametrize("group", [0, 32, 128, 256])
@pytest.mark.parametrize("res", [None, BF, F32])
def test_codes(P, T, d, group, res):
    x, w = integers(T, d, T + d)
    r = None if res is None else integers(T, d, d, dtype=res)[0]
    check(P, x, w.to(BF), r, group)
    check(P, x, (w * 2.0 ** -3).float(), r, group)


@pytest.mark.parametrize("T,d", [(5, 41), (700, 333), (300, 1001), (700, 4099), (3, 20001)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_codes_of_rows_on_no_boundary(P, T, d, group):
    x, w = integers(T, d, T + d, pad=3)
    check(P, x, w.to(BF), None, group, rows_of=d + 3)
    check(P, x, w.float(), integers(T, d, d, pad=1, dtype=F32)[0], group, rows_of=d + 2)


@pytest.mark.parametrize("e", [-120, -112, -100, -90, -80, 60, 100, 118])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("d", [512, 1001])
def test_codes_of_small_and_large_values(P, e, group, d):
    """Scales down to the smallest one there is, where an fp32 product's remainder has no place left, and up to infinity."""
    x, w = integers(9, d, d + e)
    x[3, ::3] *= -0.0
    check(P, x, (w * 2.0 ** e).float(), None, group)
    w[5] = 3e38
    check(P, x, w.float(), None, group)
