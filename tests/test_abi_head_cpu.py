"""Refusals of the head operators that need no GPU: every call below fails the library's
host validation before anything is launched."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def native():
    from semi_structured_sparse_prune24_gb300 import _native
    return _native


FAKE = 0x10000  # never dereferenced


def score(native, **kw):
    a = dict(T=4, V=100, k=0, dtype=native.P24_BF16, temperature=1.0, logits=FAKE, ldz=100, tokens=FAKE, logp=FAKE)
    return native.lib.p24_token_logprobs(C.byref(native.p24_logprobs_args(**{**a, **kw})), None)


def dscore(native, **kw):
    a = dict(T=4, V=100, dtype=native.P24_F32, temperature=1.0, logits=FAKE, ldz=100, tokens=FAKE, stats=FAKE,
             dlogp=FAKE, dlogits=2 * FAKE, ldd=100)
    return native.lib.p24_token_logprobs_bwd(C.byref(native.p24_logprobs_args(**{**a, **kw})), None)


def distill(native, bwd=False, **kw):
    a = dict(T=4, V=100, K=8, dtype=native.P24_BF16, temperature=1.0, flags=0, logits=FAKE, ldz=100, top_idx=FAKE,
             top_val=FAKE, kl=FAKE, stats=FAKE)
    if bwd:
        a.update(dkl=FAKE, dlogits=2 * FAKE, ldd=100)
    f = native.lib.p24_distill_topk_bwd if bwd else native.lib.p24_distill_topk
    return f(C.byref(native.p24_distill_args(**{**a, **kw})), None)


def test_token_logprobs_refusals(native):
    INV, ALIGN, UNS = native.P24_EINVAL, native.P24_EALIGN, native.P24_EUNSUPPORTED
    assert native.lib.p24_token_logprobs(None, None) == INV
    for kw in (dict(dtype=2), dict(T=-1), dict(V=0), dict(logits=None), dict(ldz=99), dict(tokens=None),
               dict(k=-1), dict(k=3), dict(k=3, top_idx=FAKE), dict(top_idx=FAKE, top_logp=FAKE),
               dict(logp=None), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=1e5),
               dict(temperature=float("nan"))):
        assert score(native, **kw) == INV, kw
    for kw in (dict(logits=FAKE + 1), dict(logits=FAKE + 2, dtype=native.P24_F32), dict(tokens=FAKE + 2),
               dict(logp=FAKE + 1), dict(entropy=FAKE + 2), dict(stats=FAKE + 3)):
        assert score(native, **kw) == ALIGN, kw
    for kw in (dict(V=2 ** 30 + 1, ldz=2 ** 31), dict(k=native.P24_TOPK_MAX + 1, top_idx=FAKE, top_logp=FAKE)):
        assert score(native, **kw) == UNS, kw
    assert score(native, T=0, logits=None) == 0  # no rows: nothing to do, nothing launched


def test_token_logprobs_bwd_refusals(native):
    INV, ALIGN = native.P24_EINVAL, native.P24_EALIGN
    assert native.lib.p24_token_logprobs_bwd(None, None) == INV
    for kw in (dict(stats=None), dict(tokens=None), dict(dentropy=FAKE), dict(dlogits=None), dict(ldd=99),
               dict(dlogits=FAKE, ldd=104), dict(temperature=2e4)):
        assert dscore(native, **kw) == INV, kw
    for kw in (dict(dlogits=2 * FAKE + 2), dict(stats=FAKE + 2), dict(dlogp=FAKE + 2)):
        assert dscore(native, **kw) == ALIGN, kw
    assert dscore(native, T=0) == 0


def test_distill_refusals(native):
    INV, ALIGN, UNS = native.P24_EINVAL, native.P24_EALIGN, native.P24_EUNSUPPORTED
    assert native.lib.p24_distill_topk(None, None) == INV
    assert native.lib.p24_distill_topk_bwd(None, None) == INV
    for bwd in (False, True):
        for kw in (dict(flags=2), dict(K=-1), dict(top_idx=None), dict(top_val=None), dict(dce=FAKE), dict(ce=FAKE),
                   dict(ldz=50), dict(temperature=1e-5)):
            assert distill(native, bwd, **kw) == INV, (bwd, kw)
        for kw in (dict(K=native.P24_TOPK_MAX + 1), dict(V=2 ** 19 + 1, ldz=2 ** 20, flags=native.P24_DISTILL_TAIL)):
            assert distill(native, bwd, **kw) == UNS, (bwd, kw)
        assert distill(native, bwd, top_idx=FAKE + 2) == ALIGN
        assert distill(native, bwd, T=0) == 0
    assert distill(native, kl=None) == INV
    assert distill(native, dkl=FAKE) == INV                      # weights, but no gradient to write
    assert distill(native, True, stats=None) == INV
    assert distill(native, True, dlogits=FAKE, ldd=128) == INV   # in place needs the same stride
    assert distill(native, True, dlogits=2 * FAKE + 1) == ALIGN
