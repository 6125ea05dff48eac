"""The operators around the sparse FFN chained on one stream without host syncs, launched with programmatic
stream serialization: bit-identical to the same calls with a synchronisation after each; captured and replayed; and with
scratch that an earlier call of another size has left full."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def P():
    import semi_structured_sparse_prune24_gb300 as P
    yield P
    assert P.p24_query_status() == 0


def chain(P, tok, E, w, sync=lambda: None):
    T, (V, d) = tok.shape[0], E.shape
    out = []

    def note(*ts):
        out.extend(ts)
        sync()
    x = P.p24_embed(tok, E, scale=8.0)
    note(x)
    a = P.p24_rmsnorm(x, w)
    note(a["y"], a["rstd"])
    b = P.p24_rmsnorm(a["y"], w, residual=x)
    note(b["y"], b["h"], b["rstd"])
    q = P.p24_rmsnorm(b["h"], w, group=64)
    note(q["scale"], q["y"].view(torch.uint8))
    v = P.p24_dequant8(q["y"], q["scale"], 64)
    note(v)
    g = P.p24_rmsnorm_bwd(v, b["h"], w, b["rstd"], dres=b["y"])
    note(g["dx"], g["dweight"])
    h = P.p24_rmsnorm_bwd(g["dx"], x, w, a["rstd"], dres=g["dx"])
    note(h["dx"], h["dweight"])
    dE = P.p24_embed_bwd(h["dx"], tok, V, scale=8.0)
    note(dE)
    grads = [dE, g["dweight"], h["dweight"]]
    scaled = [torch.empty_like(t) for t in grads]
    n = P.p24_clip_grads(grads, 0.5, out=scaled)
    note(n, *scaled)
    P.p24_embed_bwd(h["dx"], tok, V, scale=-8.0, dW=dE, accumulate=True)
    note(dE.clone(), P.p24_grad_norm([dE]))
    return out


def data(T, V, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tok = (torch.rand(T, generator=g, device="cuda") ** 2 * V).to(torch.int32)
    return tok, (torch.randn((V, d), generator=g, device="cuda") * 0.02).to(BF), 1 + 0.1 * torch.randn(d, generator=g, device="cuda")


@pytest.mark.parametrize("T,V,d", [(1, 50, 64), (300, 1000, 767), (5000, 3000, 1024)])
def test_chain(P, T, V, d):
    a = data(T, V, d, T)
    want = chain(P, *a, sync=torch.cuda.synchronize)
    for _ in range(5):
        got = chain(P, *a)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_sizes_in_turn_and_captured(P):
    sizes = [data(700, 900, 512, 1), data(40, 5000, 1001, 2)]
    want = [chain(P, *a, sync=torch.cuda.synchronize) for a in sizes]
    bufs = [[t.clone() for t in a] for a in sizes]
    graphs, outs = [], []
    for b in bufs:                                   # two graphs, each with scratch of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(P, *b))
        graphs.append(g)
    for k in (0, 1, 1, 0, 1):
        graphs[k].replay()
    for k in (1, 0):                                 # both at once
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graphs[k].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(o, w))


def test_two_streams_at_once(P):
    sizes = [data(3000, 900, 2048, 3), data(2000, 5000, 1001, 4)]
    want = [chain(P, *a, sync=torch.cuda.synchronize) for a in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [None, None]
    for _ in range(3):
        for k, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[k] = chain(P, *sizes[k])
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(o, w))


def test_tables_gradients_back_to_back(P):
    """A table's gradient read, scaled, written by another kernel and made again, without a wait on the host between: its
    zeros overtake nothing that came before them, and what comes after finds the sums."""
    g = torch.Generator(device="cuda").manual_seed(11)
    V, d = 40000, 1000
    dW = torch.empty((V, d), dtype=torch.bfloat16, device="cuda")
    runs = []
    for T in (1, 300, 5000):
        tok = torch.randint(0, V, (T,), generator=g, device="cuda").int()
        dY = torch.randn((T, d), generator=g, device="cuda").bfloat16()
        table = P.p24_embed_bwd(dY, tok, V)
        torch.cuda.synchronize()
        norm = P.p24_grad_norm([table])
        clipped = table.clone()
        P.p24_clip_grads([clipped], 1.0)
        torch.cuda.synchronize()
        runs.append((tok, dY, table, norm, clipped))
    got = []
    for k in range(30):
        tok, dY = runs[k % 3][:2]
        P.p24_embed_bwd(dY, tok, V, dW=dW)
        got.append((P.p24_grad_norm([dW]), P.p24_embed(tok, dW), P.p24_clip_grads([dW], 1.0), P.p24_embed(tok, dW)))
        if k % 7 == 3:
            dW.fill_(float("nan"))
        elif k % 7 == 5:
            P.p24_rmsnorm(dY, None, out={"y": dW[:len(dY)]})
    torch.cuda.synchronize()
    for k, (norm, rows, again, scaled) in enumerate(got):
        tok, _, table, want, clipped = runs[k % 3]
        assert torch.equal(norm, want) and torch.equal(again, want)
        assert torch.equal(rows, table[tok.long()]) and torch.equal(scaled, clipped[tok.long()])
