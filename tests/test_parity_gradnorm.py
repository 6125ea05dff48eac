"""GPU parity of p24_grad_norm and p24_clip_grads against the fp64 oracle (oracle/block_oracle.py).

Tolerances, u = 2^-24: a thread adds the squares of at most 128 elements in fp32 (130u relative on a sum of positive
terms), the rest is pairs of fp32 numbers or fp64 (less than u in all); on the norm half of it, and its rounding: 70u. A
scaled gradient: 70u, the quotient,
the product, and the output's rounding: (73u + half a step) |g|."""
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


def check(P, grads, max_norm, out=None):
    before = [f64(t) for t in grads]
    n, want = BO.clip(before, max_norm)
    norm = P.p24_grad_norm(grads)
    got = P.p24_clip_grads(grads, max_norm, out=out)
    assert torch.equal(norm, got)
    assert abs(float(got) - n) <= 70 * U * n
    for k, (t, w) in enumerate(zip(grads if out is None else out, want)):
        if n <= max_norm * (1 - 100 * U):
            assert np.array_equal(f64(t), before[k])
        e = torch.finfo(t.dtype).eps / 2
        assert (np.abs(f64(t) - w) <= (73 * U + e) * np.abs(w) + TINY[t.dtype]).all(), k
        if out is not None and t.data_ptr() != grads[k].data_ptr():
            assert np.array_equal(f64(grads[k]), before[k])


SETS = {
    "one element": [(1, F32, 0)],
    "a vector": [(768, F32, 0)],
    "odd sizes and starts": [(1, BF, 1), (7, BF, 3), (8, BF, 0), (0, F32, 0), (1001, BF, 5), (4099, F32, 1), (17, F32, 3), (30000, BF, 7)],
    "chunk ends": [(16384, BF, 0), (16385, BF, 0), (8192, F32, 0), (8191, F32, 0), (16391, BF, 1), (8195, F32, 1), (3 * 16384 + 2, BF, 2)],
    "17 tensors": [(100 + k, BF if k % 3 else F32, k % 4) for k in range(17)],
    "129 tensors": [(1 + 31 * k, BF if k % 2 else F32, 0) for k in range(129)],
    "2000 tensors": [(1 + k % 50, BF if k % 5 else F32, k % 2) for k in range(2000)],
    "a matrix": [(3000 * 1001, BF, 0), (0, BF, 0), (1001, F32, 0)],
}


def make(spec, seed, sigma=1e-2):
    rng = np.random.default_rng(seed)
    ts = []
    for n, dt, off in spec:
        full = torch.full((n + off + 8,), float("nan"), dtype=dt, device="cuda")
        full[off:off + n] = torch.as_tensor(rng.normal(size=n) * sigma, device="cuda").to(dt)
        ts.append(full[off:off + n])
    return ts


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_clip_in_place(P, name, max_norm):
    check(P, make(SETS[name], 1), max_norm)


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_clip_into_other_tensors(P, name, max_norm):
    out = make([(n, dt, (off + 1) % 4) for n, dt, off in SETS[name]], 2)
    grads = make(SETS[name], 1)
    check(P, grads, max_norm, out)
    mixed = [g if k % 2 else o for k, (g, o) in enumerate(zip(grads, out))]
    check(P, grads, max_norm, mixed)


@pytest.mark.parametrize("sigma", [1e-30, 1e-20, 1e15, 1e25, 1e36])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sizes_whose_squares_leave_fp32(P, sigma, dt):
    check(P, make([(20000, dt, 1), (5, dt, 0)], 3, sigma), sigma)


def test_small_beside_large(P):
    a, b = make([(20000, F32, 0)], 4, 1e-25) + make([(3, F32, 1)], 5, 1e-24)
    check(P, [a, b], 1e-26)
    a[7] = 1e20
    check(P, [a, b], 1e20)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 5, 9999])
def test_a_norm_that_is_not_finite_scales_nothing(P, bad, at):
    grads = make([(10000, BF, 1), (33, F32, 0)], 6)
    grads[0][at] = bad
    before = [t.clone() for t in grads]
    out = [torch.zeros_like(t) for t in grads]
    n = P.p24_clip_grads(grads, 1e-3, out=out)
    assert not np.isfinite(float(n)) and np.isnan(float(n)) == np.isnan(bad)
    P.p24_clip_grads(grads, 1e-3)
    for t, o, b in zip(grads, out, before):
        assert torch.equal(t.nan_to_num(7), b.nan_to_num(7)) and torch.equal(o.nan_to_num(7), b.nan_to_num(7))


def test_zeros_and_empty_tensors(P):
    z = torch.zeros(5000, device="cuda")
    assert float(P.p24_clip_grads([z, torch.empty(0, device="cuda")], 1.0)) == 0 and bool((z == 0).all())
    assert float(P.p24_grad_norm([torch.empty(0, dtype=BF, device="cuda")])) == 0
    assert float(P.p24_clip_grads([torch.empty((0, 4), device="cuda")], 1.0)) == 0


def test_shapes_do_not_matter(P):
    g = torch.randn((30, 41), device="cuda")
    assert torch.equal(P.p24_grad_norm([g]), P.p24_grad_norm([g.view(-1)]))
    assert torch.equal(P.p24_grad_norm([g]), P.p24_grad_norm([g.t()]))
    with pytest.raises(ValueError):
        P.p24_grad_norm([g[:, :40]])


def test_a_model(P):
    """Tens of millions of elements in full, against torch in fp64, twice the same."""
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.empty(n, device="cuda", dtype=dt).normal_(0, 1e-3, generator=g)
             for n, dt in ((30_000_001, BF), (12345, F32), (17_000_000, F32), (1, BF))]
    n = float(torch.stack([t.double().square().sum() for t in grads]).sum().sqrt())
    out = [torch.empty_like(t) for t in grads]
    norm = P.p24_clip_grads(grads, 1.0, out=out)
    assert abs(float(norm) - n) <= 70 * U * n and torch.equal(norm, P.p24_grad_norm(grads))
    for t, o in zip(grads, out):
        w = t.double() / n
        e = torch.finfo(t.dtype).eps / 2
        assert bool(((o.double() - w).abs() <= (73 * U + e) * w.abs() + TINY[t.dtype]).all())
    again = [torch.empty_like(t) for t in grads]
    P.p24_clip_grads(grads, 1.0, out=again)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_scratch_norm_and_another_stream(P):
    grads = make(SETS["17 tensors"], 7)
    want = P.p24_grad_norm(grads)
    ws = torch.full((int(P.lib.p24_grad_norm_workspace_size(17)),), 255, dtype=torch.uint8, device="cuda")
    n = torch.empty(1, device="cuda")
    assert P.p24_grad_norm(grads, norm=n, workspace=ws) is n and torch.equal(n, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = P.p24_clip_grads(grads, 1e-3, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals_of_the_binding(P):
    g = [torch.ones(5, device="cuda")]
    for call, err in ((lambda: P.p24_grad_norm([]), ValueError), (lambda: P.p24_grad_norm([g[0].double()]), TypeError),
                      (lambda: P.p24_clip_grads(g, 0.0), P.P24Error), (lambda: P.p24_clip_grads(g, float("inf")), P.P24Error),
                      (lambda: P.p24_clip_grads(g, 1.0, out=[]), ValueError),
                      (lambda: P.p24_clip_grads(g, 1.0, out=[torch.ones(4, device="cuda")]), P.P24Error),
                      (lambda: P.p24_grad_norm(g, norm=torch.ones(2, device="cuda")), ValueError),
                      (lambda: P.p24_grad_norm(g, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), P.P24Error)):
        with pytest.raises(err):
            call()


def test_a_tensor_listed_twice(P):
    """Counted twice by the norm; refused where it would be scaled twice, or written while it is read."""
    buf = torch.ones(64, device="cuda")
    a, b, c = buf[:32], buf[32:], torch.ones(32, device="cuda")
    n = float(P.p24_grad_norm([a, b, a]))
    assert abs(n - 96 ** 0.5) <= 70 * U * n
    for grads, out in (([a, b, a], None), ([b, buf[31:33]], None), ([a, c], [c, b]), ([a, b], [c, c]), ([a], [buf[1:33]])):
        with pytest.raises(ValueError, match="overlap"):
            P.p24_clip_grads(grads, 1.0, out=out)
    assert bool((buf == 1).all()) and bool((c == 1).all())
    n = P.p24_clip_grads([a, b, torch.empty(0, device="cuda"), buf[:0]], 1.0)     # neighbours and empty ones are apart
    assert float(n) == 8.0 and bool((buf == 0.125).all())
    n = P.p24_clip_grads([a, a], 1.0, out=[c, torch.empty_like(c)])               # read twice
    assert float(n) == 1.0


def test_dense_tensors_in_another_order(P):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((33, 70), generator=g, device="cuda")
    want = P.p24_grad_norm([x])
    assert torch.equal(P.p24_grad_norm([x.t()]), want)
    o = torch.empty((33, 70), device="cuda").t()
    P.p24_clip_grads([x.t()], 1.0, out=[o])
    y = x.clone()
    P.p24_clip_grads([y], 1.0)
    assert torch.equal(o, y.t())
    for bad in (x[:, :69], x[::2], x.expand(2, 33, 70)):
        with pytest.raises(ValueError):
            P.p24_grad_norm([bad])
    with pytest.raises(ValueError, match="strides"):
        P.p24_clip_grads([x.t()], 1.0, out=[torch.empty((70, 33), device="cuda")])
    with pytest.raises(TypeError):
        P.p24_clip_grads([x], None)


@pytest.mark.parametrize("e", [40, 47])
def test_many_sums_at_the_upper_end(P, e):
    """2^34 elements of 2^e (a tensor of 2 GB listed 16 times): the sum of squares passes fp32's range for e = 47. Powers
    of two, so every sum is exact."""
    x = torch.full((1 << 30,), 2.0 ** e, dtype=BF, device="cuda")
    assert float(P.p24_grad_norm([x] * 16)) == 2.0 ** (e + 17)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("given", [False, True])
def test_long_lists(P, dt, given):
    """More than 80 MB, of tensors that end inside chunks, lie at odd offsets and are empty: clipped in place and into
    others, with a place for the norm and through the C call without one."""
    import ctypes as C
    from semi_structured_sparse_prune24_gb300 import _native as N
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = torch.randn(40_000_000 if dt == F32 else 60_000_000, generator=g, device="cuda").to(dt)
    cuts = [0, 1, 12, 5000, 5001, 2_000_003, 2_000_003, 20_000_000, 20_000_017, flat.numel()]
    grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    want = float(flat.double().square().sum().sqrt())
    f = 0.25
    out = [torch.empty_like(t) for t in grads]
    if given:
        norm = P.p24_clip_grads(grads, 0.25 * want, out=out)
        assert abs(float(norm) - want) <= 70 * U * want
        f = 0.25 * want / float(norm)
    else:
        ws = torch.empty(int(N.lib.p24_grad_norm_workspace_size(len(grads))), dtype=torch.uint8, device="cuda")
        lists = [(N.p24_tensor * len(ts))(*[N.p24_tensor(t.data_ptr(), t.numel(), N.P24_F32 if dt == F32 else N.P24_BF16) for t in ts])
                 for ts in (grads, out)]
        rc = N.lib.p24_clip_grads(C.addressof(lists[0]), C.addressof(lists[1]), len(grads), 0.25 * want, None, ws.data_ptr(),
                                  ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
    e = torch.finfo(dt).eps / 2
    for t, o in zip(grads, out):
        w = t.double() * f
        assert bool(((o.double() - w).abs() <= (75 * U + e) * w.abs() + TINY[dt]).all())
    P.p24_clip_grads(grads, 0.25 * want)
    assert all(torch.equal(t, o) for t, o in zip(grads, out))
