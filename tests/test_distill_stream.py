"""DistillHead and DistillStep on a stream that is not torch's current one: what a call drops when it
returns, while its kernels are still queued, is not handed to the current stream's next allocations."""
import pytest
import torch

from synth24 import normal_bf16

pytestmark = pytest.mark.gpu

M, D, FFN, V, K = 512, 256, 1024, 2048, 16


def inputs():
    g = dict(X=normal_bf16((M, D), 1.0, 9, 1, "cuda"), W_up=normal_bf16((FFN, D), 0.06, 9, 2, "cuda"),
             W_down=normal_bf16((D, FFN), 0.06, 9, 3, "cuda"), W_head=normal_bf16((V, D), 0.3, 9, 4, "cuda"))
    g.update(b_up=torch.linspace(-0.1, 0.1, FFN, device="cuda"), b_down=torch.linspace(-0.2, 0.2, D, device="cuda"))
    g.update(labels=torch.arange(M, dtype=torch.int32, device="cuda") * 3, dkl=torch.full((M,), 1.0, device="cuda"),
             dce=torch.full((M,), 0.5, device="cuda"))
    return g


@pytest.mark.parametrize("tail,tau", [(True, 1.0), (False, 2.0)])
@pytest.mark.parametrize("raw", [False, True])
def test_dropped_intermediates_stay_the_streams_own(tail, tau, raw):
    """The side stream is held up for some milliseconds, so that every kernel of the step is still to
    come when run returns; the current stream then allocates and overwrites far more memory than the
    step's intermediates took. raw: the stream as a handle. db_up is summed by atomics, so it is
    compared up to the order of fp32 additions: 512 of them, 2^-15 of the largest; all else bit for bit."""
    import semi_structured_sparse_prune24_gb300 as P
    from semi_structured_sparse_prune24_gb300.distill import DistillHead, DistillStep
    a = inputs()
    t = DistillHead(M, D, V).teacher_list(normal_bf16((M, D), 1.0, 9, 5, "cuda"), a["W_head"], K, temperature=tau)
    a.update(top_idx=t["top_idx"], top_logp=t["top_logp"], tail=tail, temperature=tau)
    step = DistillStep(M, D, FFN, V)
    want = {n: x.clone() for n, x in step.run(**a).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = step.run(**a, stream=side.cuda_stream if raw else side)
        junk = [torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
                for rows, cols in 4 * [(M, FFN), (M, D), (FFN, D), (M, V)]]
        junk += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 14, 1 << 18, 1 << 20)]
        torch.cuda.synchronize()
        assert set(got) == set(want)
        for n in want:
            if n == "db_up":
                assert (got[n] - want[n]).abs().max() <= 2.0 ** -15 * want[n].abs().max()
            else:
                assert torch.equal(got[n], want[n]), n
        del junk, got
    assert P.p24_query_status() == 0


def test_head_calls_on_a_side_stream():
    """A list, a score and a step of the head, each on a held-up side stream, against the current stream."""
    from semi_structured_sparse_prune24_gb300.distill import DistillHead
    a = inputs()
    head, Y = DistillHead(M, D, V), a["X"]
    side = torch.cuda.Stream()
    results = []
    for s in (None, side):
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)
        t = head.teacher_list(Y, a["W_head"], K, temperature=2.0, stream=s)
        o = head.score(Y, a["W_head"], a["labels"], stream=s)
        u = head.step(Y, a["W_head"], t["top_idx"], t["top_logp"], a["dkl"], a["labels"], a["dce"], temperature=2.0,
                      tail=False, stream=s)
        junk = [torch.full((M, K), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        results.append([x.clone() for r in (t, o, u) for x in r.values()])
        del junk
    assert all(torch.equal(x, y) for x, y in zip(*results))
