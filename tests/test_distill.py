"""DistillHead and DistillStep: the head's products and the loss together, and a whole step of a
2:4 student against its dense teacher."""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO
from oracle import prune24_oracle as O
from synth24 import normal_bf16
from tests.conftest import bits_of
from tests.p24_testutil import assert_close, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    return P


def test_head_step_matches_its_pieces(P):
    """The list of a teacher head, then loss and gradients of a student head: kl against the
    oracle on the logits as stored, dY and dW against products of the stored gradient."""
    from semi_structured_sparse_prune24_gb300.distill import DistillHead
    M, d, V, K = 264, 256, 5000, 16
    Yt, Wt = normal_bf16((M, d), 1.0, 1, 1, "cuda"), normal_bf16((V, d), 0.15, 1, 2, "cuda")
    Y, W = normal_bf16((M, d), 1.0, 1, 3, "cuda"), normal_bf16((V, d), 0.15, 1, 4, "cuda")
    head = DistillHead(M, d, V)
    t = head.teacher_list(Yt, Wt, K)
    teacher = head.logits.double().cpu().numpy()
    ref = HO.token_logprobs(teacher, None, K)
    assert np.array_equal(t["top_idx"].cpu().numpy(), ref["top_idx"])
    np.testing.assert_allclose(t["top_logp"].double().cpu(), ref["top_logp"], atol=1e-4)
    labels = torch.randint(0, V, (M,), dtype=torch.int32, device="cuda")
    w = torch.full((M,), 1.0, device="cuda")
    logits = P.p24_gemm_nt(Y, W)
    o = head.step(Y, W, t["top_idx"], t["top_logp"], w, labels, 0.5 * w)
    torch.cuda.synchronize()
    assert P.p24_query_status() == 0
    want = HO.distill(logits.double().cpu().numpy(), t["top_idx"].cpu().numpy(), t["top_logp"].cpu().numpy(),
                      labels.cpu().numpy(), 1.0, True, np.ones(M), 0.5 * np.ones(M))
    np.testing.assert_allclose(o["kl"].double().cpu(), want["kl"], rtol=1e-4)
    np.testing.assert_allclose(o["ce"].double().cpu(), want["ce"], rtol=1e-4)
    D = head.logits                                     # the gradient, where the logits were
    np.testing.assert_allclose(D.double().cpu(), want["dlogits"], rtol=2 ** -7, atol=1e-6)
    assert_close(o["dY"], O.dense_nt(bits_of(D), np.ascontiguousarray(bits_of(W).T))[0], "dY")
    assert_close(o["dW"], O.dense_tn(bits_of(D), bits_of(Y))[0], "dW")
    s = head.score(Y, W, labels)
    np.testing.assert_allclose(-s["logp"].double().cpu(), want["ce"], rtol=1e-4)


def test_student_learns_from_its_teacher(P):
    """Plain gradient steps on the weights of a 2:4 student bring its divergence from the dense
    teacher it was copied from down; the masks hold 2 of 4 throughout."""
    from semi_structured_sparse_prune24_gb300.distill import DistillHead, DistillStep
    M, d, ffn, V, K = 512, 256, 512, 2048, 32
    X = normal_bf16((M, d), 1.0, 3, 1, "cuda")
    W_up, W_down = normal_bf16((ffn, d), 0.06, 3, 2, "cuda"), normal_bf16((d, ffn), 0.06, 3, 3, "cuda")
    W_head = normal_bf16((V, d), 0.3, 3, 4, "cuda")
    b_up, b_down = torch.zeros(ffn, device="cuda"), torch.zeros(d, device="cuda")
    Yt = (torch.relu(X.float() @ W_up.float().T) @ W_down.float().T).bfloat16()        # the dense teacher
    t = DistillHead(M, d, V).teacher_list(Yt, W_head, K)
    step = DistillStep(M, d, ffn, V)
    w = torch.full((M,), 1.0 / M, device="cuda")
    up, down = W_up.float(), W_down.float()
    losses = []
    for _ in range(30):
        o = step.run(X, up.bfloat16(), b_up, down.bfloat16(), b_down, W_head, t["top_idx"], t["top_logp"], w)
        losses.append(o["kl"].mean().item())
        up -= 0.5 * o["dW_up"].float()
        down -= 0.5 * o["dW_down"].float()
        b_up -= 0.5 * o["db_up"]
        b_down -= 0.5 * o["db_down"]
    assert P.p24_query_status() == 0
    assert all(np.isfinite(losses)) and losses[-1] < 0.8 * losses[0], losses
    nz = (f32(o["dW_up"]) != 0).reshape(ffn, d // 4, 4).sum(-1)
    assert nz.max() <= 2


def test_head_refuses_a_vocabulary_off_the_products_grid():
    from semi_structured_sparse_prune24_gb300.distill import DistillHead
    with pytest.raises(ValueError):
        DistillHead(8, 64, 5001)
