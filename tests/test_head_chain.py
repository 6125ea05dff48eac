"""The head's row operators stay ordered in a user's stream.

They are launched like the library's other kernels: one may start while the stream's previous
kernel still runs, and waits on the device for its completion before its first global access.
A teacher's list, a student's loss and gradient, the gradient alone and a score are chained with
torch kernels that rewrite their inputs and outputs in between, with no host synchronisation, and
have to be bit-identical to the same calls with a device synchronize after each one."""
import pytest
import torch

from synth24 import normal_bf16

pytestmark = pytest.mark.gpu


def _chain(P, teacher, student, labels, w, sync):
    def step():
        if sync:
            torch.cuda.synchronize()

    z, zt = student.clone(), teacher.clone()
    kept = []
    for i in range(3):
        t = P.p24_token_logprobs(zt, labels, k=12); step()
        zt.mul_(0.75)                       # torch rewrites an input of the previous call
        o = P.p24_distill_topk(z, t["top_idx"], t["top_logp"], labels, tail=True, dkl=w, dce=w); step()
        kept.append(t["top_idx"].clone())
        t["top_idx"].fill_(-1)              # and the list that it read
        z.sub_(o["dlogits"].to(z.dtype))
        s = P.p24_token_logprobs(z, labels, k=0); step()
        dz = P.p24_token_logprobs_bwd(z, labels, s["stats"], w, s["entropy"], w); step()
        s["stats"].zero_()
        o["dlogits"].zero_()                # outputs of earlier calls
        t2 = P.p24_token_logprobs(zt, k=7); step()
        o2 = P.p24_distill_topk(z, t2["top_idx"], t2["top_logp"], tail=False); step()
        dk = P.p24_distill_topk_bwd(z, t2["top_idx"], t2["top_logp"], o2["stats"], tail=False, dkl=w); step()
        z.add_(dk, alpha=-1.0).add_(dz, alpha=0.5)
        kept += [t["top_logp"], t["logp"], s["logp"], o["kl"], o["ce"], s["entropy"], dz, t2["top_idx"], o2["kl"], dk, z.clone()]
    torch.cuda.synchronize()
    return kept


@pytest.mark.parametrize("side_stream", [False, True])
@pytest.mark.parametrize("T,V,dtype", [(3, 30011, torch.float32), (700, 1001, torch.bfloat16), (900, 20000, torch.bfloat16)])
def test_chain_without_sync_matches_synchronised_chain(T, V, dtype, side_stream):
    import semi_structured_sparse_prune24_gb300 as P
    teacher = normal_bf16((T, V), 3.0, 51, 0, "cuda").to(dtype)
    student = normal_bf16((T, V), 3.0, 51, 1, "cuda").to(dtype)
    labels = (torch.arange(T, dtype=torch.int32, device="cuda") * 7919) % V
    w = torch.linspace(0.25, 2.0, T, device="cuda")
    ref = _chain(P, teacher, student, labels, w, sync=True)
    s = torch.cuda.Stream() if side_stream else torch.cuda.current_stream()
    with torch.cuda.stream(s):
        for _ in range(3):                  # back to back, so that launches overlap their predecessors
            got = _chain(P, teacher, student, labels, w, sync=False)
            for i, (a, b) in enumerate(zip(got, ref)):
                assert torch.isfinite(b.float()).all(), i
                assert torch.equal(a, b), i
    assert P.p24_query_status() == 0
