"""Outputs whose memory is shared with a lazy copy (torch._lazy_clone: copied when one of the two is written): the call
writes to memory of its own, and the other tensor keeps its values, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def data(d=264):
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return rnd(40, d).to(BF), rnd(40, d).to(BF), rnd(d), torch.randint(-1, 50, (40,), generator=g, device="cuda").int()


def calls(P):
    """Name, tensors that are written, and the call on them; those that are also read come with their values."""
    x, r, w, tok = data()
    o = P.p24_rmsnorm(x, w, residual=r, group=64)
    b = P.p24_rmsnorm(x, w, residual=r)
    e = lambda t: torch.zeros_like(t)  # noqa: E731
    table = torch.randn((50, 264), device="cuda")
    return [
        ("norm", [e(b["y"]), e(b["h"]), e(b["rstd"])], lambda y, h, s: P.p24_rmsnorm(x, w, residual=r, out=dict(y=y, h=h, rstd=s))),
        ("stream in place", [r.clone()], lambda h: P.p24_rmsnorm(x, w, residual=h, out=dict(h=h))),
        ("codes", [torch.zeros((40, 264), dtype=torch.uint8, device="cuda"), e(o["scale"])],
         lambda y, s: P.p24_rmsnorm(x, w, residual=r, group=64, out=dict(y=y.view(E4), scale=s))),
        ("gradient", [e(x), e(w)], lambda dx, dw: P.p24_rmsnorm_bwd(r, b["h"], w, b["rstd"], out=dict(dx=dx, dweight=dw))),
        ("gradient in place", [r.clone()], lambda dy: P.p24_rmsnorm_bwd(dy, b["h"], w, b["rstd"], out=dict(dx=dy))),
        ("values", [e(x)], lambda y: P.p24_dequant8(o["y"], o["scale"], 64, out=y)),
        ("lookup", [e(x)], lambda y: P.p24_embed(tok, table, out=y)),
        ("table", [e(table)], lambda dW: P.p24_embed_bwd(x, tok, 50, dW=dW)),
        ("table, added", [table.clone()], lambda dW: P.p24_embed_bwd(x, tok, 50, dW=dW, accumulate=True)),
        ("clip", [r.clone(), w.clone()], lambda a, c: P.p24_clip_grads([a, c], 0.5)),
        ("clip into others", [e(r), e(w), torch.zeros(1, device="cuda")], lambda a, c, n: P.p24_clip_grads([r, w], 0.5, out=[a, c], norm=n)),
        ("clip, one in place", [r.clone(), e(w)], lambda a, c: P.p24_clip_grads([a, w], 0.5, out=[a, c])),
        ("norm of gradients", [torch.zeros(1, device="cuda")], lambda n: P.p24_grad_norm([r, w], norm=n)),
    ]


def test_lazy_copies_keep_their_values(P):
    wrong = []
    for name, tensors, call in calls(P):
        want = [t.clone() for t in tensors]
        call(*want)
        before = [t.clone() for t in tensors]
        copies = [torch._lazy_clone(t) for t in tensors]
        call(*copies)
        torch.cuda.synchronize()
        if not all(torch.equal(t, b) for t, b in zip(tensors, before)):
            wrong.append(name + ": the other tensor changed")
        if not all(torch.equal(c, v) for c, v in zip(copies, want)):
            wrong.append(name + ": the result differs")
    assert not wrong, wrong
