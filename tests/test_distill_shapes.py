"""DistillHead and DistillStep hold buffers of fixed sizes: inputs of other sizes are refused before
anything is launched. On the CPU: the refusal comes before a tensor's device matters."""
import pytest
import torch

from semi_structured_sparse_prune24_gb300.distill import DistillHead, DistillStep

M, D, FFN, V, K = 16, 32, 64, 40, 4


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("rows,vocab,name", [(M + 1, V, "Y"), (M - 1, V, "Y"), (M, V + 8, "W"), (M, V - 8, "W")])
def test_head_refuses_other_sizes(rows, vocab, name):
    """More rows would be written past the logits' buffer, fewer would leave an earlier call's rows in the result."""
    head = DistillHead(M, D, V, device="cpu")
    Y, W = t(rows, D), t(vocab, D)
    idx, val, w = t(M, K, dtype=torch.int32), t(M, K, dtype=torch.float32), t(M, dtype=torch.float32)
    for call in (lambda: head.teacher_list(Y, W, K), lambda: head.score(Y, W, t(rows, dtype=torch.int32)),
                 lambda: head.step(Y, W, idx, val, w)):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            call()


@pytest.mark.parametrize("name,shape", [("dY", (M, D + 8)), ("dY", (M - 1, D)), ("dW", (V - 8, D)), ("dW", (V, D - 8))])
def test_head_refuses_outputs_of_other_sizes(name, shape):
    head = DistillHead(M, D, V, device="cpu")
    idx, val, w = t(M, K, dtype=torch.int32), t(M, K, dtype=torch.float32), t(M, dtype=torch.float32)
    with pytest.raises(ValueError, match=f"^{name} must be"):
        head.step(t(M, D), t(V, D), idx, val, w, out={name: t(*shape)})


@pytest.mark.parametrize("name,shape", [("X", (M + 1, D)), ("X", (M, D - 8)), ("W_up", (FFN + 8, D)), ("b_up", (FFN - 8,)),
                                        ("W_down", (D, FFN + 8)), ("b_down", (D - 8,)), ("W_head", (V + 8, D))])
def test_step_refuses_other_sizes(name, shape):
    step = DistillStep(M, D, FFN, V, device="cpu")
    a = dict(X=t(M, D), W_up=t(FFN, D), b_up=t(FFN, dtype=torch.float32), W_down=t(D, FFN), b_down=t(D, dtype=torch.float32),
             W_head=t(V, D), top_idx=t(M, K, dtype=torch.int32), top_logp=t(M, K, dtype=torch.float32),
             dkl=t(M, dtype=torch.float32))
    a[name] = torch.zeros(shape, dtype=a[name].dtype)
    with pytest.raises(ValueError, match=f"^{name} must be"):
        step.run(**a)
