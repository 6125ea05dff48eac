"""Scratch that the binding allocates for a call on a stream that is not torch's current one, and drops
when the call returns with its kernels still queued: the current stream's next allocations do not get it."""
import pytest
import torch

from synth24 import FFNWorkload, ffn_inputs, normal_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    return P


def held_up():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some milliseconds
    return side


def overwrite(nbytes):
    """More than nbytes of the current stream's memory, in blocks down to a small fraction of it."""
    junk, n = [], nbytes
    while n >= 512:
        junk += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        n //= 2
    return junk


def test_column_sums(P):
    G = normal_bf16((4096, 1024), 1.0, 3, 1, "cuda")
    want = P.p24_colsum(G)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    for _ in range(2):
        out.zero_()
        P.p24_colsum(G, out, stream=held_up())
        junk = overwrite(int(P.lib.p24_colsum_workspace_size(4096, 1024)))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk


def test_ffn_step(P):
    """All but db_up, which is summed by atomics, bit for bit."""
    i = ffn_inputs(FFNWorkload("scratch", 256, 256, 512, 0.05), seed=1, device="cuda", bias=True)
    a = (i["X"], i["W_up"], i["b_up"], i["W_down"], i["b_down"], i["dY"])
    want = P.ffn24_step(*a)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    torch.cuda.synchronize()
    for _ in range(2):
        P.ffn24_step(*a, out=out, stream=held_up())
        junk = overwrite(P.ffn24_workspace_size(256, 256, 512))
        torch.cuda.synchronize()
        for n in want:
            assert n == "db_up" or torch.equal(out[n], want[n]), n
        del junk
    assert P.p24_query_status() == 0
