"""GPU parity of p24_rmsnorm, p24_rmsnorm_bwd and p24_dequant8 against the fp64 oracle (oracle/block_oracle.py).

Tolerances, derived for u = 2^-24 (half a step of fp32 is u relative, of bf16 2^-8, of e4m3 2^-4):
  * h is x + r rounded once in fp32 and once to r's type, the oracle's once: equal, or for bf16 one step apart where
    the fp32 sum lies at a midpoint. The norm of the GPU's own h is what the oracle is then given.
  * The sum of squares adds positive terms, at most 128 in a thread and 10 joins: 140u relative; mean, eps and
    the reciprocal square root 8u; on rstd half of the first: e = 80u.
  * y: two products more, then its own rounding: (e + 2u + half a step) |y|.
  * 8 bits: the scale is off by (e + 6u) relative; a code is the nearest one to a value off by (2e + 12u): it is one of
    those that the oracle's value times 1 -+ 2^-15 (512u) rounds to. Values are then code * scale rounded to bf16.
  * The gradient's mean c of d terms p = dy xh w is off by (140u + 2e + 4u) mean|p|; with g = dy w,
    dx by rstd (4u |g| + |xh| (2e + 6u) |c| + |xh| 306u mean|p|) + e |dx - dres| + 2u (|dres| + |dx|), then rounded.
  * dw: each term off by e + 3u, and at most T / 152 + 64 additions on a term's way: (T / 152 + 150) u sum|dy xh|.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO

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


def f64(t):
    return t.detach().double().cpu().numpy()


def half(dt):
    return torch.finfo(dt).eps / 2


def mat(a, dtype, pad=0, off=0):
    """[T, d] values as a view with row stride d + pad that starts `off` elements into its memory; NaN around it."""
    T, d = a.shape
    full = torch.full((T * (d + pad) + off + 8,), float("nan"), dtype=dtype, device="cuda")
    v = full[off:off + T * (d + pad)].view(T, d + pad)[:, :d] if T else full[:0].view(0, d)
    v.copy_(torch.as_tensor(np.ascontiguousarray(a), device="cuda"))
    return v


def close(got, want, bound, name):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), name
    bound = np.broadcast_to(bound, want.shape)
    bad = np.abs(got[fin] - want[fin]) > bound[fin]
    assert not bad.any(), (name, int(bad.sum()), got[fin][bad][:4], want[fin][bad][:4], bound[fin][bad][:4])


def stream(T, d, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, d)) * np.exp(0.7 * rng.normal(size=(T, 1)))
    x[:, rng.random(d) < 0.01] *= 25
    return x, rng


def check_norm(P, x, w, r, y_dtype, group, eps=1e-6, out=None):
    res = P.p24_rmsnorm(x, w, residual=r, eps=eps, group=group, out=out if out is not None else
                        ({} if y_dtype in (None, E4) else {"y": torch.empty(x.shape, dtype=y_dtype, device="cuda")}))
    h = f64(x)
    if r is not None:
        want = (x.double() + r.double()).cpu().numpy()
        fin = np.isfinite(want)
        step = half(r.dtype) * np.abs(want) + U * np.abs(want) + TINY[r.dtype]
        close(res["h"], np.where(fin, want, want), np.where(fin, step, 0), "h")
        h = f64(res["h"])
    _, rstd, y = BO.rmsnorm(h, None if w is None else f64(w), eps=eps)
    close(res["rstd"], rstd, E * rstd + 2.0 ** -149, "rstd")
    if group is None:
        close(res["y"], y, (E + 2 * U + half(res["y"].dtype)) * np.abs(y) + TINY[res["y"].dtype], "y")
        return res
    s = BO.scales(y, group)
    close(res["scale"], s, (E + 6 * U) * s, "scale")
    v = y / BO.spread(s, y.shape[1], group)
    q, lo, hi = f64(res["y"].float()), BO.round_e4m3(v * (1 - 2.0 ** -15)), BO.round_e4m3(v * (1 + 2.0 ** -15))
    fin = np.isfinite(v)
    assert np.array_equal(np.isnan(q), np.isnan(v))
    assert ((q == lo) | (q == hi))[fin].all()
    vals = P.p24_dequant8(res["y"], res["scale"], group)
    want = q * BO.spread(f64(res["scale"]), y.shape[1], group)
    close(vals, want, (half(BF) + U) * np.abs(want) + TINY[BF], "values")
    out32 = P.p24_dequant8(res["y"], res["scale"], group, out=torch.empty(x.shape, dtype=F32, device="cuda"))
    close(out32, want, U * np.abs(want) + TINY[F32], "values in fp32")
    return res


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 64), (5, 255), (17, 256), (1, 1000), (9, 1024), (4, 1025), (7, 2049), (1, 4096), (3, 5001),
          (2, 8192), (1, 8199), (2, 16384), (1, 32768), (2, 32761), (700, 768), (2500, 96), (5000, 17)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("kind", [(BF, None, None), (BF, BF, BF), (BF, F32, BF), (F32, BF, F32), (F32, F32, None)])
def test_norm(P, T, d, kind):
    dx, dr, dw = kind
    a, rng = stream(T, d, T * 1000 + d)
    x = mat(a, dx)
    r = None if dr is None else mat(stream(T, d, d)[0], dr)
    w = None if dw is None else torch.as_tensor(1 + 0.2 * rng.normal(size=d), device="cuda").to(dw)
    check_norm(P, x, w, r, None, None)


@pytest.mark.parametrize("T,d", [(1, 40), (3, 333), (5, 1000), (2, 2048), (4, 4999), (300, 512), (2, 20000)])
@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 0), (0, 1), (5, 3), (8, 4)])
def test_norm_strides_and_alignments(P, T, d, y_dtype, pad, off):
    a, rng = stream(T, d, d + pad)
    x, r = mat(a, BF, pad, off), mat(rng.normal(size=(T, d)), F32, pad, (off * 3) % 8)
    w = torch.as_tensor(1 + 0.2 * rng.normal(size=d + off), device="cuda").to(BF)[off:]
    out = dict(y=mat(a, y_dtype, pad + 1, off), h=mat(a, F32, 2 * pad, 1))
    check_norm(P, x, w, r, None, None, out=out)


@pytest.mark.parametrize("T,d", [(1, 1), (3, 31), (2, 32), (5, 257), (4, 1000), (3, 4096), (2, 5001), (300, 512), (1, 32768)])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("pad", [0, 3])
def test_norm_8_bits(P, T, d, group, pad):
    a, rng = stream(T, d, d + group)
    x, r = mat(a, BF, pad), mat(rng.normal(size=(T, d)), BF, pad)
    w = torch.as_tensor(1 + 0.2 * rng.normal(size=d), device="cuda").float()
    n = -(-d // group) if group else 1
    buf = torch.zeros(T * (d + pad), dtype=torch.uint8, device="cuda").view(E4).view(T, d + pad)
    out = dict(y=buf[:, :d], scale=mat(np.zeros((T, n)), F32, pad))
    check_norm(P, x, w, r, E4, group, out=out)
    assert bool((buf.view(torch.uint8)[:, d:] == 0).all())  # columns past the row are left as they were


def test_norm_rows_at_the_edge_of_the_type(P):
    """Zeros, a group of zeros, NaN, infinities, squares beyond fp32, and the smallest numbers."""
    d = 300
    a = np.random.default_rng(0).normal(size=(10, d))
    a[0] = 0
    a[1, 64:192] = 0
    a[2, 5] = np.nan
    a[3, 7] = np.inf
    a[4, 9] = -np.inf
    a[5] *= 1e30
    a[6] *= 3e37
    a[7] *= 1e-30
    a[8] = 2.0 ** -133
    a[9, 1:] = 0
    a[9, 0] = 3e38
    w = torch.full((d,), 1.5, device="cuda")
    for dt in (BF, F32):
        for group in (None, 0, 64):
            check_norm(P, mat(a, dt), w, None, None, group)
            check_norm(P, mat(a, dt), None, mat(np.zeros_like(a), dt), None, group, eps=1e-12)


def test_norm_in_place(P):
    a, rng = stream(40, 1000, 1)
    w = torch.ones(1000, device="cuda")
    x, r = mat(a, BF), mat(rng.normal(size=(40, 1000)), F32)
    want = P.p24_rmsnorm(x, w, residual=r)
    r2 = r.clone()
    got = P.p24_rmsnorm(x, w, residual=r2, out={"h": r2})          # the stream itself
    assert got["h"] is r2 and torch.equal(r2, want["h"]) and torch.equal(got["y"], want["y"])
    x2 = x.clone()
    got = P.p24_rmsnorm(x2, w, residual=r, out={"y": x2})          # the branch becomes the normed rows
    assert torch.equal(x2, want["y"]) and torch.equal(got["h"], want["h"])
    rb = r.to(BF)
    want = P.p24_rmsnorm(x, w, residual=rb)
    x2, r2 = x.clone(), rb.clone()
    P.p24_rmsnorm(x2, w, residual=r2, out={"h": x2, "y": r2})
    assert torch.equal(x2, want["h"]) and torch.equal(r2, want["y"])


def check_bwd(P, dy, h, w, dres, dx_dtype=None, out=None, eps=1e-6):
    H, D, W = f64(h), f64(dy), None if w is None else f64(w)
    R = None if dres is None else f64(dres)
    rstd = 1 / np.sqrt((H * H).mean(1) + eps)
    rs = torch.as_tensor(rstd, device="cuda").float()
    o = P.p24_rmsnorm_bwd(dy, h, w, rs, dres=dres, dweight=True, out=out if out is not None else
                          ({} if dx_dtype is None else {"dx": torch.empty(h.shape, dtype=dx_dtype, device="cuda")}))
    dx, dw = BO.rmsnorm_bwd(D, H, W, eps, R)
    rc, xh = rstd[:, None], H * rstd[:, None]
    g = D if W is None else D * W
    p = np.abs(g * xh).mean(1, keepdims=True)
    c = np.abs((g * xh).mean(1, keepdims=True))
    own = np.abs(dx - (0 if R is None else R))
    b = rc * (4 * U * np.abs(g) + np.abs(xh) * (2 * E + 6 * U) * c + np.abs(xh) * 306 * U * p) + E * own
    b = b + 2 * U * (np.abs(dx) + (0 if R is None else np.abs(R)))
    dt = o["dx"].dtype
    close(o["dx"], dx, b + half(dt) * (np.abs(dx) + b) + TINY[dt], "dx")
    T = len(H)
    close(o["dweight"], dw, (T / 152 + 150) * U * np.abs(D * xh).sum(0) + TINY[F32], "dweight")
    return o


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("kind", [(BF, BF, BF, BF), (BF, F32, None, F32), (F32, BF, F32, BF), (F32, F32, BF, None)])
def test_norm_gradient(P, T, d, kind):
    th, td, tr, tw = kind
    a, rng = stream(T, d, T + d)
    h, dy = mat(a, th), mat(rng.normal(size=(T, d)) * 1e-2, td)
    dres = None if tr is None else mat(rng.normal(size=(T, d)) * 1e-2, tr)
    w = None if tw is None else torch.as_tensor(1 + 0.2 * rng.normal(size=d), device="cuda").to(tw)
    check_bwd(P, dy, h, w, dres, dx_dtype=BF if T % 2 else F32)


@pytest.mark.parametrize("T,d", [(1, 40), (3, 333), (5, 1000), (2, 2048), (4, 4999), (700, 512), (2, 20001)])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (5, 3), (8, 4)])
def test_norm_gradient_strides_and_alignments(P, T, d, pad, off):
    a, rng = stream(T, d, d + pad)
    h, dy = mat(a, BF, pad, off), mat(rng.normal(size=(T, d)), F32, pad + 1, (3 * off) % 8)
    dres = mat(rng.normal(size=(T, d)), BF, 2 * pad, 1)
    w = torch.as_tensor(1 + 0.2 * rng.normal(size=d + off), device="cuda").float()[off:]
    check_bwd(P, dy, h, w, dres, out={"dx": mat(a, BF, pad, off)})


def test_norm_gradient_in_place(P):
    a, rng = stream(33, 520, 4)
    h, dy, dres = mat(a, BF), mat(rng.normal(size=(33, 520)), BF), mat(rng.normal(size=(33, 520)), BF)
    w = torch.ones(520, device="cuda")
    rs = torch.as_tensor(1 / np.sqrt((f64(h) ** 2).mean(1)), device="cuda").float()
    want = P.p24_rmsnorm_bwd(dy, h, w, rs, dres=dres)
    for which in (0, 1, 2):
        ts = [dy.clone(), h.clone(), dres.clone()]
        got = P.p24_rmsnorm_bwd(ts[0], ts[1], w, rs, dres=ts[2], out={"dx": ts[which]})
        assert torch.equal(ts[which], want["dx"]) and torch.equal(got["dweight"], want["dweight"])


def test_no_rows(P):
    w = torch.ones(64, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    o = P.p24_rmsnorm(x, w, residual=x)
    assert o["y"].shape == (0, 64) and o["rstd"].shape == (0,)
    g = torch.full((64,), 7.0, device="cuda")
    o = P.p24_rmsnorm_bwd(x, x, w, torch.empty(0, device="cuda"), out={"dweight": g})
    assert o["dx"].shape == (0, 64) and bool((g == 0).all())
    assert P.p24_dequant8(x.to(E4), torch.empty((0, 1), device="cuda")).shape == (0, 64)


def test_without_weight_gradient(P):
    a, rng = stream(5, 64, 2)
    h, dy = mat(a, BF), mat(rng.normal(size=(5, 64)), BF)
    rs = torch.ones(5, device="cuda")
    assert set(P.p24_rmsnorm_bwd(dy, h, None, rs)) == {"dx"}
    assert set(P.p24_rmsnorm_bwd(dy, h, torch.ones(64, device="cuda"), rs, dweight=False)) == {"dx"}


@pytest.mark.parametrize("d", [777, 4096])
def test_repeated_calls_are_bit_identical(P, d):
    a, rng = stream(3000, d, 5)
    x, r, dy = mat(a, BF), mat(a[::-1], BF), mat(rng.normal(size=(3000, d)), BF)
    w = torch.as_tensor(1 + 0.2 * rng.normal(size=d), device="cuda").float()
    one, two = (P.p24_rmsnorm(x, w, residual=r) for _ in range(2))
    assert all(torch.equal(one[k], two[k]) for k in one)
    back = [P.p24_rmsnorm_bwd(dy, one["h"], w, one["rstd"], dres=r) for _ in range(2)]
    assert all(torch.equal(back[0][k], back[1][k]) for k in back[0])


def test_a_training_batch_in_full(P):
    """More rows than CTAs many times over, against torch in fp64 on the GPU."""
    T, d = 12000, 2056
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r, dy, dres = (torch.randn((T, d), generator=g, device="cuda").to(BF) for _ in range(4))
    w = torch.randn(d, generator=g, device="cuda") * 0.1 + 1
    o = P.p24_rmsnorm(x, w, residual=r)
    h = o["h"].double()
    assert torch.equal(o["h"], (x.float() + r.float()).to(BF))
    rstd = 1 / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    y = h * rstd * w.double()
    assert bool(((o["y"].double() - y).abs() <= (E + 2 * U + half(BF)) * y.abs()).all())
    b = P.p24_rmsnorm_bwd(dy, o["h"], w, o["rstd"], dres=dres)
    xh, gg = h * rstd, dy.double() * w.double()
    dx = dres.double() + rstd * (gg - xh * (gg * xh).mean(1, keepdim=True))
    slack = rstd * (4 * U * gg.abs() + xh.abs() * 500 * U * (gg * xh).abs().mean(1, keepdim=True)) + 100 * U * (dx.abs() + dres.double().abs())
    assert bool(((b["dx"].double() - dx).abs() <= slack + half(BF) * (dx.abs() + slack)).all())
    dw = (dy.double() * xh).sum(0)
    assert bool(((b["dweight"].double() - dw).abs() <= (T / 152 + 150) * U * (dy.double() * xh).abs().sum(0)).all())


def test_another_stream(P):
    a, rng = stream(200, 768, 6)
    x, w = mat(a, BF), torch.ones(768, device="cuda")
    want = P.p24_rmsnorm(x, w, residual=x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = P.p24_rmsnorm(x, w, residual=x, stream=s)
    back = P.p24_rmsnorm_bwd(got["y"], got["h"], w, got["rstd"], stream=s)
    s.synchronize()
    assert torch.equal(got["y"], want["y"])
    want = P.p24_rmsnorm_bwd(want["y"], want["h"], w, want["rstd"])
    assert all(torch.equal(back[k], want[k]) for k in back)


def test_refusals_of_the_binding(P):
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    for kw, err in ((dict(weight=torch.ones(63, device="cuda")), ValueError), (dict(weight=w.double()), TypeError),
                    (dict(residual=x[:3]), ValueError), (dict(residual=x.double()), TypeError), (dict(group=48), P.P24Error),
                    (dict(out={"y": x[:, :32]}), ValueError), (dict(group=0, out={"y": x.clone()}), TypeError),
                    (dict(residual=x, out={"h": x.float()}), TypeError), (dict(eps=0.0), P.P24Error),
                    (dict(out={"rstd": torch.zeros(3, device="cuda")}), ValueError)):
        with pytest.raises(err):
            P.p24_rmsnorm(x, **kw)
    with pytest.raises(ValueError):
        P.p24_rmsnorm(torch.zeros((64, 4), dtype=BF, device="cuda").t(), w)
    with pytest.raises(P.P24Error):
        P.p24_rmsnorm_bwd(x, x, w, torch.ones(4, device="cuda"), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("d", [4, 130, 520, 4096, 4099, 20000])
@pytest.mark.parametrize("sx,sw", [(1e15, 1e25), (1e-5, 1e-36), (1e25, 1e10), (1e-3, 1e-3), (3e-20, 1.0)])
def test_row_scales_where_products_with_the_weight_leave_fp32(P, d, sx, sw):
    """The scale of a whole row is found from h w before the norm is known, where that is representable. The scale within
    that of the values, E + 6u; a code is one of those that the value times 1 -+ 2^-15 rounds to."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((3, d), generator=g, device="cuda") * sx
    x[1] = 0
    w = torch.randn(d, generator=g, device="cuda") * sw
    o = P.p24_rmsnorm(x, w, eps=1e-12, group=0)
    h = x.double()
    y = h / (h.square().mean(1, keepdim=True) + 1e-12).sqrt() * w.double()
    top = y.abs().amax(1, keepdim=True) / 448
    s = torch.where(top == 0, 1.0, top.clamp_min(2.0 ** -118))
    u = 2.0 ** -24
    assert bool(((o["scale"].double() - s).abs() <= 86 * u * s).all())
    v = y / s
    q = o["y"].float()
    near = [(v * (1 + k * 2.0 ** -15)).clamp(-448, 448).float().to(torch.float8_e4m3fn).float() for k in (-1, 1)]
    assert bool(((q == near[0]) | (q == near[1])).all())
