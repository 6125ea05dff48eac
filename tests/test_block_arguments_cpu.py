"""Arguments of the operators around the sparse FFN that the binding refuses by themselves, before it looks at the tensors
and so before anything is launched: no GPU is needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def N():
    from semi_structured_sparse_prune24_gb300 import _native
    return _native


class NoTruth:
    def __bool__(self):
        raise RuntimeError("neither true nor false")


@pytest.mark.parametrize("what", [torch.tensor([True, False]), NoTruth()])
def test_accumulate_without_a_truth_value(N, what):
    """Not taken for False, which would overwrite the gradient that the caller wants added to."""
    dY, tok = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="accumulate must be true or false"):
        N.p24_embed_bwd(dY, tok, 4, dW=torch.zeros(4, 8), accumulate=what)
