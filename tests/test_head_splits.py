"""The head's row operators where the way they are laid out changes: from one CTA a row to several,
from few rows to more than run at once, shares that end inside a stage, grids that are spread by
their shared memory. Against the fp64 oracle, with the tolerances of test_parity_head."""
import numpy as np
import pytest

from tests.test_parity_head import BF, F32, P, check_distill, check_score, dev, f64, logits, teacher_list  # noqa: F401

pytestmark = pytest.mark.gpu

# rows by vocabulary: below and above 152 and 304 CTAs, shares of 1, 2, 4 and 8
SIZES = [(1, 9001), (19, 16401), (38, 33000), (70, 9001), (152, 4101), (153, 8300), (200, 20011), (305, 12001), (460, 8999),
         (620, 8203)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("k", [0, 20, 64])
def test_score_layouts(P, dtype, T, V, k):  # noqa: F811
    z, rng = logits(T, V, dtype, T + V + k, pad=T % 3)
    z[0, V // 2:] = -float("inf")
    if T > 4:
        z[3, 7:] = -float("inf")        # fewer finite elements than alternatives
        z[4] = -float("inf")
    check_score(P, z, rng.integers(0, V, T), k, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("mode", ["step", "bwd"])
def test_distill_layouts(P, dtype, T, V, tail, mode):  # noqa: F811
    z, rng = logits(T, V, dtype, T + V, pad=T % 3)
    idx, val = teacher_list(rng, T, V, 20)
    w = f64(dev(rng.random(T) + 0.1, F32))
    check_distill(P, z, idx, val, rng.integers(0, V, T), [1.0, 2.0][T % 2], tail, w, w[::-1].copy(), mode, inplace=tail)
