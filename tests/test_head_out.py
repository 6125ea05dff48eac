"""What the head operators hand back: a result holds what the call wrote, nothing else."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    return P


def test_a_reused_dict_of_outputs_brings_nothing_stale_back(P):
    """A dict of outputs from a call that wrote more: what this call does not write is not in its result."""
    z = torch.randn((5, 777), device="cuda")
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    full = P.p24_token_logprobs(z, tok, k=4)
    part = P.p24_token_logprobs(z, k=0, entropy=False, out=full)
    assert set(part) == {"stats"} and part["stats"] is full["stats"]
    assert set(P.p24_token_logprobs(z, tok, k=4, out=full)) == set(full)
    idx, val = full["top_idx"], full["top_logp"]
    w = torch.ones(5, device="cuda")
    full = P.p24_distill_topk(z, idx, val, tok, dkl=w, dce=w)
    assert set(full) == {"kl", "ce", "stats", "dlogits"}
    assert set(P.p24_distill_topk(z, idx, val, dkl=w, out=full)) == {"kl", "stats", "dlogits"}


def test_head_step_brings_no_stale_cross_entropy_back(P):
    from semi_structured_sparse_prune24_gb300.distill import DistillHead
    Y, W = (torch.randn(s, device="cuda").bfloat16() for s in ((16, 64), (512, 64)))
    head = DistillHead(16, 64, 512)
    t = head.teacher_list(Y, W, 4)
    w, lab = torch.ones(16, device="cuda"), torch.zeros(16, dtype=torch.int32, device="cuda")
    full = head.step(Y, W, t["top_idx"], t["top_logp"], w, lab, w)
    assert "ce" in full
    kept = {n: full[n] for n in ("kl", "ce", "stats", "dY", "dW")}
    assert "ce" not in head.step(Y, W, t["top_idx"], t["top_logp"], w, out=kept)
