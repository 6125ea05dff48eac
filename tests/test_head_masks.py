"""Rows of logits masked by a finite value: alternatives where fewer entries are left than asked for."""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO
from tests.test_parity_head import BF, F32, P, f64  # noqa: F401

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
