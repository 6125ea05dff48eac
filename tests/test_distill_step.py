"""Every result of DistillStep.run against the oracles: the FFN's gradients against the oracle's step on
the dY that the head's products give, the head's against products of the logits' gradient, and that
gradient and the losses against the head's own operator and oracle."""
import numpy as np
import pytest
import torch

from oracle import head_oracle as HO
from oracle import prune24_oracle as O
from synth24 import FFNWorkload, normal_bf16
from tests.conftest import bits_of
from tests.p24_testutil import assert_close
from tests.test_parity_ffn import compare_step, oracle_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("with_labels", [False, True])
def test_step_against_the_oracles(tail, tau, with_labels):
    import semi_structured_sparse_prune24_gb300 as P
    from semi_structured_sparse_prune24_gb300.distill import DistillHead, DistillStep
    M, d, ffn, V, K = 264, 256, 512, 2000, 24
    X, Yt = normal_bf16((M, d), 1.0, 21, 1, "cuda"), normal_bf16((M, d), 1.0, 21, 2, "cuda")
    W_up, W_down = normal_bf16((ffn, d), 0.08, 21, 3, "cuda"), normal_bf16((d, ffn), 0.08, 21, 4, "cuda")
    W_head = normal_bf16((V, d), 0.3, 21, 5, "cuda")
    b_up, b_down = torch.linspace(-0.3, 0.3, ffn, device="cuda"), torch.linspace(0.4, -0.4, d, device="cuda")
    t = DistillHead(M, d, V).teacher_list(Yt, W_head, K, temperature=tau)
    w = torch.linspace(0.5, 1.5, M, device="cuda")
    labels = (torch.arange(M, dtype=torch.int32, device="cuda") * 53) % V if with_labels else None
    c = 0.5 * w if with_labels else None
    step = DistillStep(M, d, ffn, V)
    o = step.run(X, W_up, b_up, W_down, b_down, W_head, t["top_idx"], t["top_logp"], w, labels, c, tau, tail)
    assert set(o) == {"kl", "stats", "dlogits", "dW_head", "db_up", "db_down", "dX", "dW_up", "dW_down"} | (
        {"ce"} if with_labels else set())

    # what the step does not hand out, by the same calls: they are deterministic
    H = P.spmm24_fwd(X, step.up, b_up, relu=True)
    Y = P.spmm24_fwd(H, step.down, b_down)
    logits = P.p24_gemm_nt(Y, W_head)
    values = t["top_logp"] if tail else t["top_logp"] * tau
    h = P.p24_distill_topk(logits, t["top_idx"], values, labels, tau, tail, w, c)
    assert torch.equal(h["dlogits"], o["dlogits"]) and torch.equal(h["kl"], o["kl"])
    dY = P.p24_gemm_nt(h["dlogits"], W_head.t().contiguous())
    dH = P.spmm24_bwd_dx(dY, step.down_T, gate=H)
    torch.cuda.synchronize()
    assert P.p24_query_status() == 0

    assert_close(logits, O.dense_nt(bits_of(Y), bits_of(W_head))[0], "logits")
    ref = HO.distill(logits.double().cpu().numpy(), t["top_idx"].cpu().numpy(), values.cpu().numpy(),
                     None if labels is None else labels.cpu().numpy(), tau, tail)
    np.testing.assert_allclose(o["kl"].double().cpu(), ref["kl"], rtol=1e-4, atol=1e-5)
    if with_labels:
        np.testing.assert_allclose(o["ce"].double().cpu(), ref["ce"], rtol=1e-4)
    D = bits_of(o["dlogits"])
    assert_close(dY, O.dense_nt(D, np.ascontiguousarray(bits_of(W_head).T))[0], "dY")
    assert_close(o["dW_head"], O.dense_tn(D, bits_of(Y))[0], "dW_head")
    inp = dict(X=X, W_up=W_up, b_up=b_up, W_down=W_down, b_down=b_down, dY=dY)
    got = dict(H=H, Y=Y, dH=dH, **{n: o[n] for n in ("dX", "dW_up", "db_up", "dW_down", "db_down")})
    compare_step(got, oracle_step(inp, False), FFNWorkload("step", M, d, ffn, 0.08), False)
