"""Every element of every output of the operators around the sparse FFN is written, and is a number: outputs are NaN before
the call (codes: the code that is NaN), and what is compared is that all of them ARE within the tolerance, which a NaN is not.
References are the formulas in fp64 by torch on the GPU, the tolerances those derived in test_parity_norm.py and
test_parity_embed.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E = 80 * U
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TINY = {BF: 2.0 ** -134, F32: 2.0 ** -150}


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def half(dt):
    return torch.finfo(dt).eps / 2


def nan(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, want, bound, name):
    ok = (got.double() - want).abs() <= bound
    assert bool(ok.all()), (name, int((~ok).sum()), ok.numel(), got[~ok][:4], want[~ok][:4])


def test_a_nan_is_not_within():
    g = torch.tensor([1.0, float("nan")], device="cuda")
    with pytest.raises(AssertionError):
        within(g, torch.ones(2, device="cuda").double(), 1.0, "g")


def matrix(T, d, dtype, g, pad=0, scale=1.0):
    v = nan((T, d + pad), dtype)[:, :d]
    v.copy_(torch.randn((T, d), generator=g, device="cuda") * scale)
    return v


SIZES = [(1, 1), (3, 7), (9, 64), (5, 333), (400, 512), (305, 513), (20000, 40), (9000, 127), (6000, 300), (3000, 1023), (2500, 2049), (1500, 4096),
         (1500, 5001), (1200, 6290), (900, 8192), (800, 8191), (500, 12000), (300, 16384), (300, 16383), (200, 20000), (2, 32768)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("x,r,pad", [(BF, None, 0), (BF, BF, 0), (F32, None, 0), (BF, F32, 0), (BF, F32, 3)])
@pytest.mark.parametrize("group", [None, 0, 64])
def test_norm(P, T, d, x, r, pad, group):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    X, R, w = matrix(T, d, x, g, pad), None if r is None else matrix(T, d, r, g), 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    n = group or d
    out = dict(rstd=nan((T,), F32), y=nan((T, d), x))
    if r is not None:
        out["h"] = nan((T, d), r)
    if group is not None:
        out["y"] = torch.full((T, d), 0x7f, dtype=torch.uint8, device="cuda").view(E4)
        out["scale"] = nan((T, -(-d // n)), F32)
    P.p24_rmsnorm(X, w, residual=R, group=group, out=out)
    h = X.double()
    if r is not None:
        want = h + R.double()
        within(out["h"], want, (half(r) + U) * want.abs() + TINY[r], "h")
        h = out["h"].double()
    rstd = 1 / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    within(out["rstd"], rstd[:, 0], E * rstd[:, 0], "rstd")
    y = h * rstd * w.double()
    if group is None:
        return within(out["y"], y, (E + 2 * U + half(x)) * y.abs() + TINY[x], "y")
    top = torch.stack([c.abs().amax(1) for c in y.split(n, 1)], 1) / 448
    top = torch.where(top == 0, 1.0, top)
    within(out["scale"], top, (E + 6 * U) * top, "scale")
    v = y / top.repeat_interleave(n, 1)[:, :d]
    q = out["y"].float()
    near = [(v * (1 + k * 2.0 ** -15)).clamp(-448, 448).float().to(E4).float() for k in (-1, 1)]
    assert bool(((q == near[0]) | (q == near[1])).all())
    for dt in (BF, F32):
        want = q.double() * out["scale"].double().repeat_interleave(n, 1)[:, :d]
        values = P.p24_dequant8(out["y"], out["scale"], group, out=nan((T, d), dt))
        within(values, want, (half(dt) + U) * want.abs() + TINY[dt], "values")


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("h,dy,r,dx,pad", [(BF, BF, None, BF, 0), (BF, BF, BF, BF, 0), (F32, F32, F32, F32, 0), (BF, F32, BF, BF, 3)])
def test_gradient(P, T, d, h, dy, r, dx, pad):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    H, D, w = matrix(T, d, h, g, pad), matrix(T, d, dy, g, 0, 0.1), 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    R = None if r is None else matrix(T, d, r, g, 0, 0.1)
    rc = 1 / (H.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    out = dict(dx=nan((T, d), dx), dweight=nan((d,), F32))
    ws = torch.full((max(16, int(P.lib.p24_rmsnorm_bwd_workspace_size(T, d))),), 255, dtype=torch.uint8, device="cuda")  # NaN
    P.p24_rmsnorm_bwd(D, H, w, rc[:, 0].float(), dres=R, out=out, workspace=ws)
    xh, gw = H.double() * rc, D.double() * w.double()
    mean, p = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    own = rc * (gw - xh * mean)
    res = torch.zeros_like(own) if R is None else R.double()
    b = rc * (4 * U * gw.abs() + xh.abs() * (2 * E + 6 * U) * mean.abs() + xh.abs() * 306 * U * p) + E * own.abs()
    b = b + 2 * U * ((own + res).abs() + res.abs())
    within(out["dx"], own + res, b + half(dx) * ((own + res).abs() + b) + TINY[dx], "dx")
    within(out["dweight"], (D.double() * xh).sum(0), (T / 152 + 150) * U * (D.double() * xh).abs().sum(0) + TINY[F32], "dweight")


def tokens_of(kind, T, V, g):
    at = torch.arange(T, device="cuda")
    if kind == "often":
        t = (torch.rand(T, generator=g, device="cuda") ** 4 * (V + 2)).long() - 1     # padding on both sides
    elif kind == "one":
        t = torch.full_like(at, V - 1)
    elif kind == "none":
        t = torch.where(at % 2 == 0, -1, V + at)
    elif kind == "falling":
        t = (T - at) % V
    else:
        t = at // 2 % V
    return t.int()


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 513, 8), (2, 3, 5), (31, 7, 2049), (33, 600, 64), (257, 50, 100), (1024, 3000, 40), (4096, 300, 24),
                                   (4097, 1000, 33), (20000, 5000, 16), (300, 262144, 8), (2000, 9000, 1000)])
@pytest.mark.parametrize("kind", ["often", "one", "none", "falling", "pairs"])
def test_tables(P, T, V, d, kind):
    """The lookup's rows, the table's gradient, and the gradient added to a table whose other rows keep their bits."""
    dt, dw = ((BF, F32), (F32, BF), (BF, BF), (F32, F32))[(T + len(kind)) % 4]
    g = torch.Generator(device="cuda").manual_seed(T + V)
    tok = tokens_of(kind, T, V, g)
    dY = torch.randn((T, d), generator=g, device="cuda").to(dt)
    s = 0.75
    at = torch.where((tok >= 0) & (tok < V), tok, V).long()
    want, mass, n = (torch.zeros((V + 1, k), dtype=torch.float64, device="cuda") for k in (d, d, 1))
    want.index_add_(0, at, dY.double() * s)
    mass.index_add_(0, at, dY.double().abs() * s)
    n.index_add_(0, at, torch.ones((T, 1), dtype=torch.float64, device="cuda"))
    want, mass, n = want[:V], mass[:V], n[:V]
    ws = torch.full((int(P.lib.p24_embed_bwd_workspace_size(T, d)),), 255, dtype=torch.uint8, device="cuda")
    err = (n + 2) * U * mass
    dW = P.p24_embed_bwd(dY, tok, V, s, dW=nan((V, d), dw), workspace=ws)
    within(dW, want, err + half(dw) * (want.abs() + err) + TINY[dw], "dW")
    assert bool((dW[(n == 0)[:, 0]] == 0).all())
    old = torch.randn((V, d), generator=g, device="cuda").to(dw)
    ws.fill_(255)
    added = P.p24_embed_bwd(dY, tok, V, s, dW=old.clone(), accumulate=True, workspace=ws)
    err = err + U * (want + old.double()).abs()
    within(added, want + old.double(), err + half(dw) * ((want + old.double()).abs() + err) + TINY[dw], "added")
    assert torch.equal(added[(n == 0)[:, 0]], old[(n == 0)[:, 0]])
    rows = P.p24_embed(tok, old, s, out=nan((T, d), dt))
    exact = torch.cat([old.double() * s, torch.zeros((1, d), dtype=torch.float64, device="cuda")])[at]
    within(rows, exact, (U + half(dt)) * exact.abs() + TINY[dt], "rows")


@pytest.mark.parametrize("sizes", [[1], [7, 4099, 0, 17], [300000, 5], [1 + k % 90 for k in range(1000)], [25_000_000, 1001]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_clip(P, sizes, dt):
    g = torch.Generator(device="cuda").manual_seed(len(sizes))
    grads = [torch.randn(n, generator=g, device="cuda").to(dt) for n in sizes]
    want = float(torch.stack([t.double().square().sum() for t in grads]).sum().sqrt())
    out, norm = [nan((n,), dt) for n in sizes], nan((1,), F32)
    ws = torch.full((int(P.lib.p24_grad_norm_workspace_size(len(sizes))),), 255, dtype=torch.uint8, device="cuda")
    P.p24_clip_grads(grads, 0.5 * want, out=out, norm=norm, workspace=ws)
    assert abs(float(norm) - want) <= 70 * U * want
    for o, t in zip(out, grads):
        within(o, t.double() * 0.5, (73 * U + half(dt)) * 0.5 * t.double().abs() + TINY[dt], "scaled")
