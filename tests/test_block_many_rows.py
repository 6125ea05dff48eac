"""The row operators around the sparse FFN where units take many rows: rings that wrap, every width class and layout,
and matrices whose offsets pass 32 bits. References are the formulas in fp64 by torch on the GPU, which shares nothing
with the kernels; the tolerances are those derived in test_parity_norm.py, test_parity_embed.py and
test_parity_gradnorm.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
E = 80 * U
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    torch.cuda.empty_cache()
    assert P.p24_query_status() == 0


def half(dt):
    return torch.finfo(dt).eps / 2


def matrix(T, d, dtype, g, pad=0, off=0, scale=1.0):
    full = torch.empty(T * (d + pad) + off, dtype=dtype, device="cuda")
    v = full[off:].view(T, d + pad)[:, :d]
    v.copy_(torch.randn((T, d), generator=g, device="cuda") * scale)
    return v


def blocks(T, d):
    step = max(1, (1 << 25) // d)
    return [slice(t, min(T, t + step)) for t in range(0, T, step)]


def check(T, got, want, bound, name):
    bad = (got.double() - want).abs() > bound
    assert not bool(bad.any()), (name, int(bad.sum()), got[bad][:4], want[bad][:4])


def check_norm(P, x, r, w, y_dtype, group):
    T, d = x.shape
    out = {} if group is not None else {"y": torch.empty((T, d), dtype=y_dtype, device="cuda")}
    o = P.p24_rmsnorm(x, w, residual=r, group=group, out=out)
    for s in blocks(T, d):
        h = x[s].double()
        if r is not None:
            want = h + r[s].double()
            check(T, o["h"][s], want, (half(r.dtype) + U) * want.abs(), "h")
            h = o["h"][s].double()
        rstd = 1 / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
        check(T, o["rstd"][s], rstd[:, 0], E * rstd[:, 0], "rstd")
        y = h * rstd * w.double()
        if group is None:
            check(T, o["y"][s], y, (E + 2 * U + half(y_dtype)) * y.abs() + 2.0 ** -134, "y")
            continue
        n = group or d
        top = torch.stack([c.abs().amax(1) for c in y.split(n, 1)], 1) / 448
        top = torch.where(top == 0, 1.0, top)              # a group of zeros has a scale of 1
        check(T, o["scale"][s], top, (E + 6 * U) * top, "scale")
        v = y / top.repeat_interleave(n, 1)[:, :d]
        q = o["y"][s].float()
        # a code is one of those that the value times 1 -+ 2^-15 rounds to
        near = [(v * (1 + k * 2.0 ** -15)).clamp(-448, 448).float().to(E4).float() for k in (-1, 1)]
        assert bool(((q == near[0]) | (q == near[1])).all())
        vals = P.p24_dequant8(o["y"][s], o["scale"][s], group)
        want = q.double() * o["scale"][s].double().repeat_interleave(n, 1)[:, :d]
        check(T, vals, want, (half(BF) + U) * want.abs() + 2.0 ** -134, "values")


def check_bwd(P, dy, h, w, dres, dx_dtype):
    T, d = h.shape
    rstd = torch.cat([1 / (h[s].double().square().mean(1) + 1e-6).sqrt() for s in blocks(T, d)]).float()
    o = P.p24_rmsnorm_bwd(dy, h, w, rstd, dres=dres, out={"dx": torch.empty((T, d), dtype=dx_dtype, device="cuda")})
    dw, mass = torch.zeros(d, device="cuda", dtype=torch.float64), torch.zeros(d, device="cuda", dtype=torch.float64)
    for s in blocks(T, d):
        rc = rstd[s].double()[:, None]
        xh, g = h[s].double() * rc, dy[s].double() * w.double()
        mean, p = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
        own = rc * (g - xh * mean)
        r = torch.zeros_like(own) if dres is None else dres[s].double()
        b = rc * (4 * U * g.abs() + xh.abs() * (2 * E + 6 * U) * mean.abs() + xh.abs() * 306 * U * p) + E * own.abs()
        b = b + 2 * U * ((own + r).abs() + r.abs())
        check(T, o["dx"][s], own + r, b + half(dx_dtype) * ((own + r).abs() + b) + 2.0 ** -134, "dx")
        dw += (dy[s].double() * xh).sum(0)
        mass += (dy[s].double() * xh).abs().sum(0)
    check(T, o["dweight"], dw, (T / 152 + 150) * U * mass, "dweight")


SIZES = [(20000, 40), (9000, 127), (6000, 300), (5000, 512), (4000, 513), (3000, 1023), (2500, 2049), (1500, 4096), (1500, 5001),
         (1200, 6290), (900, 8192), (800, 8191), (700, 12000), (500, 16384), (400, 16383), (300, 20000)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("x,r,y", [(BF, None, BF), (BF, BF, BF), (BF, F32, BF), (F32, None, F32)])
@pytest.mark.parametrize("group", [None, 0, 128])
def test_norm(P, T, d, x, r, y, group):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    check_norm(P, matrix(T, d, x, g), None if r is None else matrix(T, d, r, g), w, y, group)


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("h,dy,r,dx", [(BF, BF, None, BF), (BF, BF, BF, BF), (BF, BF, F32, F32), (F32, F32, F32, F32)])
def test_gradient(P, T, d, h, dy, r, dx):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    check_bwd(P, matrix(T, d, dy, g, scale=0.1), matrix(T, d, h, g), w, None if r is None else matrix(T, d, r, g, scale=0.1), dx)


@pytest.mark.parametrize("T,d", [(9000, 40), (5000, 333), (3000, 1001), (1500, 4999), (600, 9000)])
@pytest.mark.parametrize("pad,off", [(3, 1), (8, 4), (5, 0)])
def test_matrices_without_common_boundaries(P, T, d, pad, off):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    check_norm(P, matrix(T, d, BF, g, pad, off), matrix(T, d, BF, g, 2 * pad, 0), w, BF, None)
    check_bwd(P, matrix(T, d, BF, g, pad + 1, off), matrix(T, d, F32, g, 2, 1), w, matrix(T, d, BF, g), BF)


@pytest.mark.parametrize("d", [32768, 16384, 8191])
def test_offsets_beyond_32_bits(P, d):
    """2.2e9 elements in each matrix; the last rows, whose offsets pass 2^31 elements, and the first."""
    T = (1 << 31) // d + 1000
    x = torch.empty((T, d), dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(d)
    for s in blocks(T, d):
        x[s] = torch.randn((s.stop - s.start, d), generator=g, device="cuda").to(BF)
    w = torch.ones(d, device="cuda")
    o = P.p24_rmsnorm(x, w, residual=x, out={"h": torch.empty_like(x)})
    back = P.p24_rmsnorm_bwd(o["y"], o["h"], w, o["rstd"], out={"dx": torch.empty_like(x)})
    for s in (slice(0, 50), slice(T // 2, T // 2 + 50), slice(T - 1000, T)):
        h = (x[s].double() * 2).to(BF).double()
        rstd = 1 / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
        check(T, o["h"][s], h, 0 * h, "h")
        check(T, o["y"][s], h * rstd, (E + 2 * U + half(BF)) * (h * rstd).abs(), "y")
        xh, dy = h * rstd, o["y"][s].double()
        dx = rstd * (dy - xh * (dy * xh).mean(1, keepdim=True))
        slack = rstd * (4 * U * dy.abs() + xh.abs() * 500 * U * (dy * xh).abs().mean(1, keepdim=True))
        check(T, back["dx"][s], dx, slack + half(BF) * (dx.abs() + slack) + 2.0 ** -134, "dx")


def test_embedding_beyond_32_bits(P):
    """A table of 2.2e9 elements, and as many looked up; the gradient of its last rows."""
    V, d = 140000, 16000
    W = torch.empty((V, d), dtype=BF, device="cuda")
    v = torch.arange(V, device="cuda", dtype=torch.float32)[:, None]
    for s in blocks(V, d):
        W[s] = ((v[s] + torch.arange(d, device="cuda")) % 251).to(BF)
    tok = torch.arange(V - 1, -1, -1, device="cuda", dtype=torch.int32)
    Y = P.p24_embed(tok, W)
    for s in (slice(0, 100), slice(V - 100, V)):
        assert torch.equal(Y[s], W[tok[s].long()])
    tok[5:] = V - 1 - tok[5:] % 7                       # few rows, the last ones of the table
    dW = P.p24_embed_bwd(Y, tok, V, dW=W)
    assert bool((dW[: V - 7] == 0).sum() >= (V - 7 - 5) * d)
    want = torch.zeros((7, d), dtype=torch.float64, device="cuda")
    n = torch.zeros(7, device="cuda")
    for s in blocks(V, d):
        on = tok[s] >= V - 7
        want.index_add_(0, (tok[s][on] - (V - 7)).long(), Y[s][on].double())
        n.index_add_(0, (tok[s][on] - (V - 7)).long(), torch.ones(int(on.sum()), device="cuda"))
    check(7, dW[V - 7:], want, ((n[:, None] + 2) * U + half(BF)) * want.abs(), "dW")


def test_a_gradient_beyond_32_bits(P):
    n = (1 << 32) + 12345
    t = torch.empty(n, dtype=BF, device="cuda").fill_(0.5)
    t[-1] = 3.0
    small = torch.full((1000,), 2.0, device="cuda")
    want = ((n - 1) * 0.25 + 9 + 4000) ** 0.5
    norm = P.p24_clip_grads([small, t], 1.0)
    assert abs(float(norm) - want) <= 70 * U * want
    f = 1 / want
    for x, v in ((t[:1000], 0.5), (t[n // 2: n // 2 + 1000], 0.5), (t[-1000:-1], 0.5), (t[-1:], 3.0), (small, 2.0)):
        e = half(x.dtype)
        assert bool(((x.double() - v * f).abs() <= (73 * U + e) * v * f).all())


@pytest.mark.parametrize("T", [300, 2441, 3001, 4000, 5003, 9725, 20001])
@pytest.mark.parametrize("d", [40, 300, 520, 1000, 4096])
def test_the_gradient_stays_in_its_scratch(P, T, d):
    """Partial sums of the weight's gradient are as many as the scratch was sized for, for every number of CTAs."""
    from semi_structured_sparse_prune24_gb300 import _native as N
    g = torch.Generator(device="cuda").manual_seed(T)
    h, dy = matrix(T, d, BF, g), matrix(T, d, BF, g)
    need, behind = N.lib.p24_rmsnorm_bwd_workspace_size(T, d), 16 * d * 4
    ws = torch.full((need + behind,), 90, dtype=torch.uint8, device="cuda")
    rstd = 1 / (h.double().square().mean(1) + 1e-6).sqrt()
    o = P.p24_rmsnorm_bwd(dy, h, torch.ones(d, device="cuda"), rstd.float(), workspace=ws[:need])
    assert bool((ws[need:] == 90).all())
    xh = h.double() * rstd[:, None]
    check(T, o["dweight"], (dy.double() * xh).sum(0), (T / 152 + 150) * U * (dy.double() * xh).abs().sum(0), "dweight")


@pytest.mark.parametrize("T", [1, 2, 9, 31, 127, 128, 129, 304, 305])
@pytest.mark.parametrize("d", [1, 8, 13, 64, 65, 500, 2049, 4096, 8191, 8192, 8193])
@pytest.mark.parametrize("h,dy,r,dx,pad,off", [(BF, BF, BF, BF, 0, 0), (F32, BF, F32, F32, 0, 0), (BF, F32, None, BF, 3, 1),
                                               (F32, F32, BF, BF, 1, 2)])
def test_the_gradient_of_few_rows(P, T, d, h, dy, r, dx, pad, off):
    """One launch for few rows, two for more."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    check_bwd(P, matrix(T, d, dy, g, pad, off, 0.1), matrix(T, d, h, g, pad, off), w,
              None if r is None else matrix(T, d, r, g, 0, 0, 0.1), dx)


@pytest.mark.parametrize("T,d", [(1, 40), (60, 2049), (128, 4096), (128, 8192), (200, 512), (3000, 1001), (1500, 4096), (600, 8191), (9000, 40)])
@pytest.mark.parametrize("where", ["h", "dy", "dres"])
def test_the_gradient_in_place(P, T, d, where):
    """dx in the place of an input, to the rounding of the same with a place of its own; dweight counts the inputs."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    m = {k: matrix(T, d, BF, g) for k in ("h", "dy", "dres")}
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    rstd = (1 / (m["h"].double().square().mean(1) + 1e-6).sqrt()).float()
    a = P.p24_rmsnorm_bwd(m["dy"], m["h"], w, rstd, dres=m["dres"])
    xh = m["h"].double() * rstd.double()[:, None]
    mass = (m["dy"].double() * xh).abs().sum(0)
    b = P.p24_rmsnorm_bwd(m["dy"], m["h"], w, rstd, dres=m["dres"], out={"dx": m[where]})
    assert b["dx"] is m[where]
    # each is off by check_bwd's bound and half a step. With |g| <= 8, rstd and mean |g xh| <= 1.5 that bound is at most
    # 1.5 (4u 8 + |xh| (166u 1.5 + 306u 1.5)) + 80u 1.5 (8 + 1.5 |xh|) + 4u 12 < 1300u (1 + |xh|)
    gap, most = (a["dx"].double() - b["dx"].double()).abs(), a["dx"].double().abs().maximum(b["dx"].double().abs())
    assert bool((gap <= 2 * (half(BF) * most + 1300 * U * (1 + xh.abs()))).all())
    check(T, b["dweight"], a["dweight"].double(), 2 * (T / 152 + 150) * U * mass, "dweight")


@pytest.mark.parametrize("T,d", [(1, 40), (300, 2049), (3000, 1001), (1500, 4096), (600, 8191), (9000, 40), (300, 20000)])
def test_the_norm_in_place(P, T, d):
    """The stream updated in place and the branch overwritten by the norm: the same bits as with places of their own."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    x, r, w = matrix(T, d, BF, g), matrix(T, d, BF, g), torch.randn(d, generator=g, device="cuda")
    a = P.p24_rmsnorm(x, w, residual=r)
    b = P.p24_rmsnorm(x, w, residual=r, out={"h": r, "y": x})
    assert b["h"] is r and b["y"] is x
    assert torch.equal(a["h"], r) and torch.equal(a["y"], x) and torch.equal(a["rstd"], b["rstd"])
