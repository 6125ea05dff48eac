"""Refusals of the operators around the sparse FFN that need no GPU: every call below fails the library's host
validation before anything is launched, or has nothing to launch."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def N():
    from semi_structured_sparse_prune24_gb300 import _native
    return _native


A = [0x10000 * i for i in range(1, 9)]  # addresses, never dereferenced
BIG = 1 << 40


def norm(N, **kw):
    a = dict(T=4, d=100, x_dtype=N.P24_BF16, r_dtype=N.P24_BF16, w_dtype=N.P24_F32, y_dtype=N.P24_BF16, eps=1e-6,
             x=A[0], ldx=100, r=A[1], ldr=100, w=A[2], h=A[3], ldh=100, y=A[4], ldy=100, rstd=A[5])
    return N.lib.p24_rmsnorm(C.byref(N.p24_rmsnorm_args(**{**a, **kw})), None)


def dnorm(N, ws=A[7], n=BIG, **kw):
    a = dict(T=4, d=100, h_dtype=N.P24_BF16, dy_dtype=N.P24_BF16, r_dtype=N.P24_BF16, dx_dtype=N.P24_BF16,
             w_dtype=N.P24_F32, h=A[0], ldh=100, dy=A[1], lddy=100, dres=A[2], ldres=100, w=A[3], rstd=A[4], dx=A[5],
             lddx=100, dw=A[6])
    return N.lib.p24_rmsnorm_bwd(C.byref(N.p24_rmsnorm_bwd_args(**{**a, **kw})), ws, n, None)


def test_rmsnorm_refusals(N):
    INV, ALIGN, UNS = N.P24_EINVAL, N.P24_EALIGN, N.P24_EUNSUPPORTED
    assert N.lib.p24_rmsnorm(None, None) == INV
    e4 = dict(y_dtype=N.P24_E4M3, scale=A[6], lds=1)
    for kw in (dict(T=-1), dict(d=0), dict(x=None), dict(y=None), dict(h=None), dict(r=None), dict(ldx=99), dict(ldr=99),
               dict(ldh=99), dict(ldy=99), dict(x_dtype=2), dict(r_dtype=2), dict(w_dtype=2), dict(y_dtype=3),
               dict(x_dtype=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=1e5),
               dict(y=A[3]),                                   # y and h in one place
               dict(h=A[1], ldh=104), dict(h=A[0], x_dtype=N.P24_F32), dict(y=A[0], ldy=104), dict(y=A[0], y_dtype=N.P24_F32),
               dict(y=A[1], y_dtype=N.P24_F32),
               dict(e4, scale=None), dict(e4, lds=0), dict(e4, group=16), dict(e4, group=-1), dict(e4, group=100),
               dict(e4, group=32, lds=3), dict(e4, y=A[0])):
        assert norm(N, **kw) == INV, kw
    for kw in (dict(x=A[0] + 1), dict(r=A[1] + 1), dict(h=A[3] + 1), dict(y=A[4] + 1), dict(w=A[2] + 2), dict(rstd=A[5] + 2),
               dict(y=A[4] + 2, y_dtype=N.P24_F32), dict(e4, scale=A[6] + 2)):
        assert norm(N, **kw) == ALIGN, kw
    assert norm(N, d=32769, ldx=40000) == UNS
    assert norm(N, T=0, x=None, y=None) == 0


def test_rmsnorm_bwd_refusals(N):
    INV, ALIGN, UNS, SPACE = N.P24_EINVAL, N.P24_EALIGN, N.P24_EUNSUPPORTED, N.P24_ENOSPACE
    assert N.lib.p24_rmsnorm_bwd(None, None, 0, None) == INV
    for kw in (dict(T=-1), dict(d=0), dict(h=None), dict(dy=None), dict(dx=None), dict(rstd=None), dict(ldh=99), dict(lddy=99),
               dict(lddx=99), dict(ldres=99), dict(h_dtype=2), dict(dy_dtype=2), dict(dx_dtype=2), dict(r_dtype=2), dict(ws=None),
               dict(reserved=1), dict(dx=A[0], lddx=104), dict(dx=A[1], dx_dtype=N.P24_F32), dict(dx=A[2], lddx=104)):
        assert dnorm(N, **kw) == INV, kw
    for kw in (dict(h=A[0] + 1), dict(dy=A[1] + 1), dict(dx=A[5] + 1), dict(rstd=A[4] + 2), dict(dw=A[6] + 1), dict(ws=A[7] + 8)):
        assert dnorm(N, **kw) == ALIGN, kw
    need = N.lib.p24_rmsnorm_bwd_workspace_size(4, 100)
    assert need >= 4 * 100 * 4 and dnorm(N, n=need - 1) == SPACE
    assert dnorm(N, d=32769, ldh=40000) == UNS
    assert dnorm(N, T=0, dw=None) == 0
    assert N.lib.p24_rmsnorm_bwd_workspace_size(0, 100) == 0 == N.lib.p24_rmsnorm_bwd_workspace_size(-1, 100)


def test_dequant8_refusals(N):
    def call(**kw):
        a = dict(T=4, d=100, y_dtype=N.P24_BF16, group=0, q=A[0], ldq=100, scale=A[1], lds=1, y=A[2], ldy=100)
        return N.lib.p24_dequant8(C.byref(N.p24_dequant8_args(**{**a, **kw})), None)
    for kw in (dict(T=-1), dict(d=0), dict(q=None), dict(scale=None), dict(y=None), dict(ldq=99), dict(ldy=99), dict(lds=0),
               dict(group=31), dict(group=32, lds=3), dict(y_dtype=2)):
        assert call(**kw) == N.P24_EINVAL, kw
    assert call(y=A[2] + 1) == N.P24_EALIGN and call(scale=A[1] + 1) == N.P24_EALIGN
    assert call(T=0) == 0


def test_embedding_refusals(N):
    INV, ALIGN, UNS = N.P24_EINVAL, N.P24_EALIGN, N.P24_EUNSUPPORTED

    def fwd(**kw):
        a = dict(T=4, V=50, d=100, w_dtype=N.P24_BF16, y_dtype=N.P24_BF16, scale=1.0, tokens=A[0], W=A[1], ldw=100, Y=A[2], ldy=100)
        return N.lib.p24_embed(C.byref(N.p24_embed_args(**{**a, **kw})), None)

    def bwd(ws=A[7], n=BIG, **kw):
        a = dict(T=4, V=50, d=100, dy_dtype=N.P24_BF16, dw_dtype=N.P24_F32, scale=1.0, tokens=A[0], dY=A[1], lddy=100, dW=A[2], lddw=100)
        return N.lib.p24_embed_bwd(C.byref(N.p24_embed_bwd_args(**{**a, **kw})), ws, n, None)

    for f in (fwd, bwd):
        for kw in (dict(T=-1), dict(V=0), dict(d=0), dict(tokens=None), dict(scale=float("inf")), dict(scale=float("nan"))):
            assert f(**kw) == INV, kw
        assert f(tokens=A[0] + 2) == ALIGN
        assert f(V=2 ** 30) == UNS and f(d=2 ** 20 + 1) == UNS
    for kw in (dict(W=None), dict(Y=None), dict(ldw=99), dict(ldy=99), dict(w_dtype=2), dict(y_dtype=2), dict(Y=A[1])):
        assert fwd(**kw) == INV, kw
    assert fwd(W=A[1] + 1) == ALIGN and fwd(Y=A[2] + 1) == ALIGN
    for kw in (dict(dY=None), dict(dW=None), dict(lddy=99), dict(lddw=99), dict(dy_dtype=2), dict(dw_dtype=2), dict(accumulate=2),
               dict(ws=None), dict(dW=A[1])):
        assert bwd(**kw) == INV, kw
    assert bwd(dW=A[2] + 2) == ALIGN and bwd(ws=A[7] + 4) == ALIGN
    assert bwd(n=N.lib.p24_embed_bwd_workspace_size(4, 100) - 1) == N.P24_ENOSPACE
    assert fwd(T=0, tokens=None, W=None, Y=None) == 0 and bwd(T=0, tokens=None, dY=None, accumulate=1) == 0


def test_gradient_list_refusals(N):
    INV, ALIGN = N.P24_EINVAL, N.P24_EALIGN

    def ts(*rows):
        return (N.p24_tensor * len(rows))(*[N.p24_tensor(*r) for r in rows])
    one = ts((A[0], 10, N.P24_BF16))
    L = N.lib

    def norm(g, n=None, out=A[1], ws=A[7], size=BIG):
        return L.p24_grad_norm(g, len(g) if n is None else n, out, ws, size, None)

    def clip(g, out=None, m=1.0, ws=A[7], size=BIG):
        return L.p24_clip_grads(g, out, len(g), m, A[1], ws, size, None)

    assert norm(None, 1) == INV and norm(one, -1) == INV and norm(one, out=None) == INV and norm(one, ws=None) == INV
    assert norm(one, out=A[1] + 2) == ALIGN and norm(one, ws=A[7] + 8) == ALIGN
    assert norm(one, size=L.p24_grad_norm_workspace_size(1) - 1) == N.P24_ENOSPACE
    for bad in ((None, 10, 0), (A[0], -1, 0), (A[0], 10, 2)):
        assert norm(ts(bad)) == INV and clip(ts(bad)) == INV
    assert norm(ts((A[0] + 1, 10, N.P24_BF16))) == ALIGN and norm(ts((A[0] + 2, 10, N.P24_F32))) == ALIGN
    assert norm(ts((A[0], 2 ** 43, 0))) == N.P24_EUNSUPPORTED
    assert norm(ts((A[0], 2 ** 41, 0), (A[0], 2 ** 41, 0), (A[0], 1, 0))) == N.P24_EUNSUPPORTED
    for m in (0.0, -1.0, float("inf"), float("nan")):
        assert clip(one, m=m) == INV
    assert clip(one, ts((A[2], 9, N.P24_BF16))) == INV and clip(one, ts((A[2], 10, N.P24_F32))) == INV
    assert clip(one, ts((None, 10, N.P24_BF16))) == INV and clip(one, ts((A[2] + 1, 10, N.P24_BF16))) == ALIGN


def test_binding_refuses_host_tensors(N):
    x, w = torch.zeros(2, 8), torch.zeros(8)
    for call in (lambda: N.p24_rmsnorm(x, w), lambda: N.p24_rmsnorm_bwd(x, x, w, torch.zeros(2)),
                 lambda: N.p24_dequant8(x.to(torch.float8_e4m3fn), torch.zeros(2, 1)),
                 lambda: N.p24_embed(torch.zeros(2, dtype=torch.int32), x), lambda: N.p24_grad_norm([x]),
                 lambda: N.p24_embed_bwd(x, torch.zeros(2, dtype=torch.int32), 4), lambda: N.p24_clip_grads([x], 1.0),
                 lambda: N.p24_grad_norm([])):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_binding_refuses_another_device(N):
    assert N._marshal.require_device(0, 0) is None
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        N._marshal.require_device(1, 0)


def test_binding_refuses_what_is_no_tensor_or_number(N):
    x = torch.zeros(2, 8)
    for call in (lambda: N.p24_rmsnorm([1.0]), lambda: N.p24_grad_norm(3), lambda: N.p24_grad_norm([1, 2]),
                 lambda: N.p24_embed(x, None), lambda: N._marshal.rmsnorm(x), lambda: N._marshal.grads()):
        with pytest.raises(TypeError):
            call()
