"""GPU parity of p24_embed and p24_embed_bwd against the fp64 oracle (oracle/block_oracle.py).

Tolerances, u = 2^-24: the lookup is one product in fp32 and the output's rounding, (u + half a step) |y|. A row of
the gradient sums n terms in fp32, in any grouping at most n roundings on a term's way, then the scale and the
output's rounding: (n + 2) u scale sum|dY| + half a step of the result (accumulated: u more of the sum)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TINY = {BF: 2.0 ** -134, F32: 2.0 ** -150}


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def half(dt):
    return torch.finfo(dt).eps / 2


def view(T, d, dtype, pad, off, fill=float("nan")):
    full = torch.full((T * (d + pad) + off + 8,), fill, dtype=dtype, device="cuda")
    return full, full[off:off + T * (d + pad)].view(T, d + pad)[:, :d]


def tokens_of(kind, T, V, rng):
    if kind == "zipf":
        t = np.minimum(np.exp(rng.random(T) * np.log(V)).astype(np.int64) - 1, V - 1)
        t[rng.random(T) < 0.1] = -1
    elif kind == "one":
        t = np.full(T, V - 1)
    elif kind == "none":
        t = rng.choice([-1, V, V + 5, -2 ** 31, 2 ** 31 - 1], T)
    elif kind == "falling":
        t = np.arange(T, 0, -1) % V
    elif kind == "pairs":
        t = np.arange(T) // 2 % V
    else:
        t = rng.integers(0, V, T)
    return t


def dev(t):
    return torch.as_tensor(t, device="cuda").to(torch.int32)


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 100, 8192), (7, 5, 3), (48, 1000, 2049), (1000, 32000, 64), (5000, 50, 130), (2, 9, 70000)])
@pytest.mark.parametrize("tw,ty", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
def test_lookup(P, T, V, d, tw, ty, pad, off):
    rng = np.random.default_rng(T + V + d)
    _, W = view(V, d, tw, pad, off)
    W.copy_(torch.as_tensor(rng.normal(size=(V, d)), device="cuda"))
    tok = tokens_of("zipf" if T > 1 else "any", T, V, rng)
    full, Y = view(T, d, ty, 2 * pad, off)
    P.p24_embed(dev(tok), W, scale=1.7, out=Y)
    want = BO.embed(tok, f64(W), float(np.float32(1.7)))
    assert (np.abs(f64(Y) - want) <= (U + half(ty)) * np.abs(want) + TINY[ty]).all()
    assert int(torch.isnan(full).sum()) == full.numel() - T * d      # nothing else is written


def test_lookup_of_padding_and_special_rows(P):
    W = torch.tensor([[1.0, float("inf")], [float("nan"), 2.0]], device="cuda")
    Y = f64(P.p24_embed(dev([0, 1, 2, -1, -2 ** 31, 2 ** 31 - 1]), W, scale=0.0))
    assert np.isnan(Y[0, 1]) and Y[0, 0] == 0 and np.isnan(Y[1, 0]) and (Y[2:] == 0).all()
    assert P.p24_embed(dev([]), W).shape == (0, 2)


def check_bwd(P, dY, tok, V, scale, dW, accumulate=False, ws=None):
    old = f64(dW) if accumulate else None
    s = float(np.float32(scale))
    want = BO.embed_bwd(f64(dY), tok, V, s, old)
    mass = BO.embed_bwd(np.abs(f64(dY)), tok, V, abs(s))
    n = BO.embed_bwd(np.ones((len(tok), 1)), tok, V)
    got = P.p24_embed_bwd(dY, dev(tok), V, scale=scale, dW=dW, accumulate=accumulate, workspace=ws)
    assert got is dW
    err = (n + 2) * U * mass + (U * np.abs(want) if accumulate else 0)
    bound = err + half(dW.dtype) * (np.abs(want) + err) + TINY[dW.dtype]
    if accumulate:  # rows without a token are not touched, bit for bit
        assert np.array_equal(f64(dW)[n[:, 0] == 0], old[n[:, 0] == 0])
    g = f64(dW)
    bad = np.abs(g - want) > bound
    assert not bad.any(), (int(bad.sum()), g[bad][:4], want[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 513, 8), (2, 3, 5), (31, 7, 2049), (33, 600, 64), (257, 50, 100), (1024, 3000, 40),
                                   (4096, 300, 24), (4097, 1000, 33), (20000, 5000, 16), (300, 262144, 8)])
@pytest.mark.parametrize("kind", ["zipf", "one", "none", "falling", "pairs", "any"])
def test_gradient(P, T, V, d, kind):
    rng = np.random.default_rng(T + V + d)
    tok = tokens_of(kind, T, V, rng)
    dt, dw = ((BF, F32), (F32, BF), (BF, BF), (F32, F32))[(T + V) % 4]
    dY = torch.as_tensor(rng.normal(size=(T, d)), device="cuda").to(dt)
    dW = torch.full((V, d), float("nan"), dtype=dw, device="cuda")
    check_bwd(P, dY, tok, V, 0.7, dW)


@pytest.mark.parametrize("T,V,d", [(1, 4, 9), (600, 100, 77), (5000, 2000, 256)])
@pytest.mark.parametrize("pad,off", [(0, 1), (8, 0), (3, 2)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dt,dw", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_gradient_strides(P, T, V, d, pad, off, accumulate, dt, dw):
    rng = np.random.default_rng(T)
    tok = tokens_of("zipf", T, V, rng)
    _, dY = view(T, d, dt, pad, off)
    dY.copy_(torch.as_tensor(rng.normal(size=(T, d)), device="cuda"))
    full, dW = view(V, d, dw, pad + 1, off)
    if accumulate:
        dW.copy_(torch.as_tensor(rng.normal(size=(V, d)), device="cuda"))
    check_bwd(P, dY, tok, V, 3.0, dW, accumulate)
    assert int(torch.isnan(full).sum()) == full.numel() - V * d


def test_gradient_without_positions(P):
    dW = torch.full((40, 24), 3.0, device="cuda")
    e = torch.empty((0, 24), device="cuda")
    P.p24_embed_bwd(e, dev([]), 40, dW=dW, accumulate=True)
    assert bool((dW == 3).all())
    P.p24_embed_bwd(e, dev([]), 40, dW=dW)
    assert bool((dW == 0).all())


def test_wide_rows_and_a_large_vocabulary(P):
    """Digits of every pass of the sort, and rows of many column chunks; against torch in fp64."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, V, d in ((3000, 1 << 21, 8), (300, 70, 20000), (70000, 131072, 32)):
        tok = (torch.rand(T, generator=g, device="cuda", dtype=torch.float64) ** 3 * V).to(torch.int32)
        dY = torch.randn((T, d), generator=g, device="cuda")
        got = P.p24_embed_bwd(dY, tok, V)
        want = torch.zeros((V, d), dtype=torch.float64, device="cuda").index_add_(0, tok.long(), dY.double())
        mass = torch.zeros((V, d), dtype=torch.float64, device="cuda").index_add_(0, tok.long(), dY.double().abs())
        n = torch.bincount(tok.long(), minlength=V)[:, None]
        assert bool(((got.double() - want).abs() <= (n + 4) * U * mass).all())
        assert torch.equal(got, P.p24_embed_bwd(dY, tok, V))          # bit-identical


def test_scratch_of_the_caller_and_another_stream(P):
    rng = np.random.default_rng(5)
    tok, dY = dev(tokens_of("zipf", 5000, 700, rng)), torch.randn((5000, 64), device="cuda")
    want = P.p24_embed_bwd(dY, tok, 700)
    ws = torch.full((int(P.lib.p24_embed_bwd_workspace_size(5000, 64)),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(P.p24_embed_bwd(dY, tok, 700, workspace=ws), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = P.p24_embed_bwd(dY, tok, 700, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(P.P24Error):
        P.p24_embed_bwd(dY, tok, 700, workspace=ws[:64])


def test_refusals_of_the_binding(P):
    W, t = torch.zeros((5, 8), device="cuda"), dev([1, 2])
    for call, err in ((lambda: P.p24_embed(t.long(), W), TypeError), (lambda: P.p24_embed(t[None], W), ValueError),
                      (lambda: P.p24_embed(t, W, out=torch.zeros((3, 8), device="cuda")), ValueError),
                      (lambda: P.p24_embed(t, W.double()), TypeError), (lambda: P.p24_embed(t, W.t()), ValueError),
                      (lambda: P.p24_embed(t, W, scale=float("nan")), P.P24Error),
                      (lambda: P.p24_embed_bwd(W, t, 5), ValueError), (lambda: P.p24_embed_bwd(W[:2], t, 0), P.P24Error),
                      (lambda: P.p24_embed_bwd(W[:2], t, 5, accumulate=True), ValueError),
                      (lambda: P.p24_embed_bwd(W[:2], t, 5, dW=W[:4]), ValueError)):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("V", [1, 63, 64, 65, 4095, 8129, 8192, 8193, 16390, 40000])
@pytest.mark.parametrize("off", [0, 1, 37, 64])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gap", [0, 3])
def test_zeros_end_where_the_table_does(P, V, off, dt, gap):
    """Tables whose first and last bytes lie anywhere between boundaries, with gaps between rows or without, and guards."""
    for T in (0, 3):
        flat = torch.full((off + V * (1 + gap) + 70,), 7.0, dtype=dt, device="cuda")
        dW = flat[off:off + V * (1 + gap)].view(V, 1 + gap)[:, :1]
        tok = torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
        P.p24_embed_bwd(torch.ones((T, 1), dtype=dt, device="cuda"), tok, V, dW=dW)
        want = torch.zeros((V, 1), dtype=dt, device="cuda")
        want[V - 1] = T
        assert torch.equal(dW, want)
        dW.fill_(7.0)
        assert bool((flat == 7.0).all())


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 127, 128, 129, 255, 1000, 2047, 2048, 2049, 4095, 4096, 4097, 8192, 20000])
@pytest.mark.parametrize("V,d", [(3, 8), (500, 9), (60000, 1), (60000, 520)])
def test_every_way_to_sort(P, T, V, d):
    """Tokens ranked by a warp each, or sorted by a cluster, by their number and the table's size. Whole numbers, whose sums
    are exact in fp32 in any order; frequent tokens, and padding on both sides."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    tok = (torch.rand(T, generator=g, device="cuda") ** 4 * (V + 2)).int() - 1
    dY = torch.randint(-8, 9, (T, d), generator=g, device="cuda").float()
    want = torch.zeros((V + 2, d), device="cuda", dtype=torch.float64)
    want.index_add_(0, tok.long() + 1, dY.double())
    want = want[1:V + 1].float()
    assert torch.equal(P.p24_embed_bwd(dY, tok, V), want)
    old = torch.randint(-8, 9, (V, d), generator=g, device="cuda").float()
    assert torch.equal(P.p24_embed_bwd(dY, tok, V, dW=old.clone(), accumulate=True), want + old)
