"""The cases that the operators around the sparse FFN are measured on, and their plain forms.

Six kinds of pass:

  norm    root-mean-square norm of the residual stream, with the branch's addition to it; the output bf16 or fp32, or 8 bits
          (e4m3) with a scale for each row or each group of columns, which is then turned into bf16 again for the products
  dnorm   its gradient, with what reaches the stream directly added to it, and the weight's gradient
  embed   rows of the embedding table, scaled
  dembed  the table's gradient, summed over the positions of each token
  gnorm   the norm over all of a model's gradients
  clip    the same, and the gradients scaled down to a largest norm

Widths are those of the FFN workloads (synth24) and odd ones; vocabularies 32000, 50257 and 131072 as for the head's
operators; token counts from one sequence being decoded to a training batch. Tokens follow Zipf's law: the most frequent
ones make up several per cent of a batch each, and most of a vocabulary is not in it.
"""
import math

import torch

own = False
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    norm = dict(op="norm", x="bf16", res="bf16", y="bf16", w="f32")
    back = dict(op="dnorm", x="bf16", dy="bf16", w="f32")
    return [
        # one sequence being decoded: all latency
        dict(norm, name="norm_1x8192", T=1, d=8192),
        # a training batch of the widest FFN
        dict(norm, name="norm_16384x8192", T=16384, d=8192),
        # activations kept in 8 bits, with a scale for 128 columns, until a bf16 product reads them
        dict(norm, name="norm8_1999x4096_g128", T=1999, d=4096, y="e4m3", group=128, w="bf16"),
        # a stream held in fp32 beside bf16 branches, and an odd width: rows that no 16-byte vector fits
        dict(norm, name="norm_1000x5001_f32", T=1000, d=5001, res="f32"),
        # the backward of the training batch, with the gradient that the skip connection brings
        dict(back, name="dnorm_16384x8192", T=16384, d=8192, res="bf16"),
        # a ragged batch whose stream and its gradient are fp32; the first norm of a model: nothing else reaches it
        dict(back, name="dnorm_777x2049_f32", T=777, d=2049, x="f32", dy="f32", res="none"),
        # the sampled tokens of a serving batch
        dict(op="embed", name="embed_48x4096", T=48, d=4096, V=32000, table="bf16", out="bf16", scale=64.0),
        # a training batch, into a stream held in fp32
        dict(op="embed", name="embed_16384x4096_f32", T=16384, d=4096, V=131072, table="bf16", out="f32", scale=1.0),
        # a short micro-batch: the table's gradient is mostly zeros
        dict(op="dembed", name="dembed_1024x2048_V32000", T=1024, d=2048, V=32000, dy="bf16", out="bf16", scale=1.0),
        # a training batch, gradients of the table in fp32 for the optimiser
        dict(op="dembed", name="dembed_16384x4096_V131072", T=16384, d=4096, V=131072, dy="bf16", out="f32", scale=64.0),
        # adapters of rank 64 beside frozen masks: 48 small fp32 tensors
        dict(op="gnorm", name="gnorm_adapters_768", d=768, ffn=2056, layers=12, V=0, r=64, dtype="f32"),
        # eight layers of the 1.3B workload's width with embedding, biases and norms: bf16 matrices and fp32 vectors
        dict(op="clip", name="clip_8x2048x8192", d=2048, ffn=8192, layers=8, V=50257, r=0, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dnorm", "dnorm", "embed", "dembed", "dembed", "gnorm", "clip", "clip"])
    if op in ("gnorm", "clip"):
        d, ffn = _spread(rng, 64, 4096), _spread(rng, 128, 8192)
        r = rng.choice([0, 0, 16, 64])
        layers = rng.randint(1, 24 if r else max(1, min(24, 2 ** 28 // (2 * d * ffn))))
        V = rng.choice([0, 32000, 50257]) if r == 0 and d <= 2048 else 0
        return dict(op=op, d=d, ffn=ffn, layers=layers, V=V, r=r, dtype="bf16" if op == "clip" and rng.random() < 0.6 else "f32")
    d = rng.choice([768, 2048, 4096, 8192]) if rng.random() < 0.4 else _spread(rng, 64, 16384)
    T = min(_spread(rng, 1, 16384), 2 ** 26 // d)
    kind = lambda p: "f32" if rng.random() < p else "bf16"  # noqa: E731
    if op == "norm":
        case = dict(op=op, T=T, d=d, x=kind(0.2), res=rng.choice(["none", "bf16", "f32"]), y=rng.choice(["bf16", "bf16", "f32", "e4m3"]), w=kind(0.5))
        if case["y"] == "e4m3":
            case["group"] = rng.choice([0, 32, 128])
        return case
    if op == "dnorm":
        return dict(op=op, T=T, d=d, x=kind(0.4), dy=kind(0.3), res=rng.choice(["none", "bf16", "f32"]), w=kind(0.5))
    V = rng.choice([32000, 50257, 131072]) if rng.random() < 0.5 else _spread(rng, 1000, 131072)
    if op == "embed":
        return dict(op=op, T=T, d=d, V=min(V, 2 ** 28 // d), table=kind(0.3), out=kind(0.3), scale=rng.choice([1.0, 64.0, 0.7]))
    return dict(op=op, T=T, d=d, V=min(V, 2 ** 28 // d), dy=kind(0.3), out=kind(0.4), scale=rng.choice([1.0, 64.0, 0.7]))


def _gradients(case):
    """Values of the matrices and of the vectors, and how many tensors of which sizes they are."""
    d, ffn, r = case["d"], case["ffn"], case["r"]
    mats, vecs = ([ffn * r, r * d, d * r, r * ffn], []) if r else ([ffn * d, d * ffn], [ffn, d, d, d])
    mats = mats * case["layers"] + ([case["V"] * d] if case["V"] else [])
    return mats, vecs * case["layers"]


def work(case):
    op = case["op"]
    if op in ("gnorm", "clip"):
        mats, vecs = _gradients(case)
        n = sum(mats) * SIZE[case["dtype"]] + sum(vecs) * 4
        return {"bytes": 2 * n + 4 if op == "clip" else n + 4, "flops": (3 if op == "clip" else 2) * (sum(mats) + sum(vecs))}
    T, d = case["T"], case["d"]
    if op == "norm":
        res = SIZE.get(case["res"], 0)
        if case["y"] == "e4m3":  # the codes, and the bf16 values they are turned into
            y = 3 * d + 4 * -(-d // (case["group"] or d))
        else:
            y = SIZE[case["y"]] * d
        return {"bytes": T * ((SIZE[case["x"]] + 2 * res) * d + y + 4) + d * SIZE[case["w"]], "flops": 5 * T * d}
    if op == "dnorm":
        return {"bytes": T * d * (2 * SIZE[case["x"]] + SIZE[case["dy"]] + SIZE.get(case["res"], 0)) + T * 4 + d * (4 + SIZE[case["w"]]), "flops": 9 * T * d}
    if op == "embed":  # of the table, no more rows than there are tokens or entries
        return {"bytes": T * (4 + d * SIZE[case["out"]]) + min(T, case["V"]) * d * SIZE[case["table"]], "flops": T * d}
    return {"bytes": T * (4 + d * SIZE[case["dy"]]) + case["V"] * d * SIZE[case["out"]], "flops": T * d}


# ------------------------------------------------------------------ inputs
def _stream(T, d, g):
    """A residual stream: tokens of differing size, and some columns far larger than the others."""
    x = torch.randn((T, d), generator=g, device="cuda")
    x.mul_(torch.exp(0.7 * torch.randn((T, 1), generator=g, device="cuda")))
    return x.mul_(torch.where(torch.rand(d, generator=g, device="cuda") < 0.003, 25.0, 1.0))


def _tokens(T, V, g):
    """Zipf's law over a shuffled vocabulary, and some padding."""
    rank = torch.exp(torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * math.log(V)).long() - 1
    tok = torch.randperm(V, generator=g, device="cuda")[rank.clamp_(0, V - 1)].to(torch.int32)
    if T >= 64:
        tok[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
    return tok


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    op = case["op"]
    st = dict(case=dict(case), op=op)
    if op in ("gnorm", "clip"):
        mats, vecs = _gradients(case)
        flat = []
        for sizes, dt in ((mats, TYPES[case["dtype"]]), (vecs, torch.float32)):
            if sizes:
                a = torch.empty(sum(sizes), device="cuda", dtype=dt)
                a.normal_(0, 2e-3, generator=g)
                flat.append((a, sizes))
        st["flat"] = [a for a, _ in flat]
        st["grads"] = [t for a, sizes in flat for t in a.split(sizes)]
        st["clipped"] = [torch.empty_like(a) for a in st["flat"]]
        st["out"] = [t for c, (_, sizes) in zip(st["clipped"], flat) for t in c.split(sizes)]
        return st
    T, d = case["T"], case["d"]
    new = lambda *shape, t="f32": torch.empty(shape, device="cuda", dtype=TYPES[t])  # noqa: E731
    if op in ("norm", "dnorm"):
        st["w"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(TYPES[case["w"]])
        st["x"] = _stream(T, d, g).to(TYPES[case["x"]])
        st["res"] = None if case["res"] == "none" else _stream(T, d, g).to(TYPES[case["res"]])
        if op == "dnorm":
            x = st["x"].float()
            st["rstd"] = (x.square().mean(1) + EPS).rsqrt()
            del x
            st["dy"] = torch.randn((T, d), generator=g, device="cuda").mul_(1e-2).to(TYPES[case["dy"]])
            if st["res"] is not None:
                st["res"].mul_(1e-2)
            st["out"] = dict(dx=new(T, d, t=case["x"]), dweight=new(d))
            return st
        st["group"] = case.get("group")
        st["out"] = dict(rstd=new(T))
        if st["res"] is not None:
            st["out"]["h"] = new(T, d, t=case["res"])
        if case["y"] == "e4m3":
            st["out"]["y"] = torch.empty((T, d), device="cuda", dtype=torch.float8_e4m3fn)
            st["out"]["scale"] = new(T, -(-d // (case["group"] or d)))
            st["values"] = new(T, d, t="bf16")
        else:
            st["out"]["y"] = new(T, d, t=case["y"])
        return st
    V = case["V"]
    st.update(V=V, scale=case["scale"], tokens=_tokens(T, V, g))
    if op == "embed":
        st["table"] = torch.empty((V, d), device="cuda", dtype=TYPES[case["table"]]).normal_(0, 0.02, generator=g)
        st["out"] = new(T, d, t=case["out"])
    else:
        st["dy"] = torch.empty((T, d), device="cuda", dtype=TYPES[case["dy"]]).normal_(0, 1e-2, generator=g)
        st["out"] = new(V, d, t=case["out"])
    return st


# ------------------------------------------------------------------ plain forms
def _norm(st):
    case = st["case"]
    h = st["x"]
    out = {}
    if st["res"] is not None:
        h = out["h"] = (h.float() + st["res"].float()).to(st["res"].dtype)
    h = h.float()
    rstd = ((h * h).mean(1) + EPS).rsqrt()
    out["rstd"] = rstd
    y = h * rstd[:, None] * st["w"].float()
    if case["y"] != "e4m3":
        out["y"] = y.to(TYPES[case["y"]])
        return out
    T, d = y.shape
    group = case["group"] or d
    n = -(-d // group)
    if n * group != d:  # the last group is short
        y = torch.cat([y, torch.zeros((T, n * group - d), device=y.device)], 1)
    y = y.view(T, n, group)
    top = y.abs().amax(2)
    scale = torch.where(top > 0, top / 448, 1.0)
    q = (y / scale[:, :, None]).to(torch.float8_e4m3fn)
    out["scale"] = scale
    out["values"] = (q.float() * scale[:, :, None]).to(torch.bfloat16).view(T, n * group)[:, :d]
    return out


def _dnorm(st):
    x, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
    xhat = x * rstd
    g = dy * st["w"].float()
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["res"] is not None:
        dx = dx + st["res"].float()
    return dict(dx=dx.to(st["x"].dtype), dweight=(dy * xhat).sum(0))


def _embed(st):
    tok = st["tokens"].long()
    rows = st["table"][tok.clamp_min(0)].float() * st["scale"]
    return torch.where((tok >= 0)[:, None], rows, 0.0).to(st["out"].dtype)


def _dembed(st):
    tok = st["tokens"].long()
    V, d = st["out"].shape
    table = torch.zeros((V + 1, d), device=tok.device)  # the last row takes the padding
    table.index_add_(0, torch.where(tok >= 0, tok, V), st["dy"].float() * st["scale"])
    return table[:V].to(st["out"].dtype)


def _gnorm(st):
    total = sum((a.float() ** 2).sum() for a in st["flat"])  # matrices and vectors: one buffer each
    return total.sqrt().reshape(1)


def _clip(st):
    norm = _gnorm(st)
    factor = (1.0 / norm).clamp_max(1.0)
    return dict(norm=norm, grads=[(a.float() * factor).to(a.dtype) for a in st["flat"]])


def run(st):
    op = st["op"]
    if own:
        import semi_structured_sparse_prune24_gb300 as P

        if op == "norm":
            o = P.p24_rmsnorm(st["x"], st["w"], residual=st["res"], eps=EPS, group=st["group"], out=st["out"])
            if st["group"] is not None:
                values = P.p24_dequant8(o.pop("y"), o["scale"], group=st["group"], out=st["values"])
                return dict(o, values=values)
            return o
        if op == "dnorm":
            return P.p24_rmsnorm_bwd(st["dy"], st["x"], st["w"], st["rstd"], dres=st["res"], out=st["out"])
        if op == "embed":
            return P.p24_embed(st["tokens"], st["table"], scale=st["scale"], out=st["out"])
        if op == "dembed":
            return P.p24_embed_bwd(st["dy"], st["tokens"], st["V"], scale=st["scale"], dW=st["out"])
        if op == "gnorm":
            return P.p24_grad_norm(st["grads"])
        return dict(norm=P.p24_clip_grads(st["grads"], 1.0, out=st["out"]), grads=st["clipped"])
    return {"norm": _norm, "dnorm": _dnorm, "embed": _embed, "dembed": _dembed, "gnorm": _gnorm, "clip": _clip}[op](st)


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3(v):
    """The nearest of the values that 4 exponent and 3 fraction bits hold, ties to even; up to 448."""
    step = torch.exp2(torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent.double() - 4)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op in ("gnorm", "clip"):
        norm = torch.stack([torch.linalg.vector_norm(a.double()) for a in st["flat"]]).pow(2).sum().sqrt()
        if op == "gnorm":
            return norm.reshape(1)
        return dict(norm=norm.reshape(1), grads=[a.double() / norm.clamp_min(1.0) for a in st["flat"]])
    if op == "embed":
        tok = st["tokens"].long()
        rows = torch.zeros((case["T"], case["d"]), device="cuda", dtype=torch.float64)
        rows[tok >= 0] = st["table"][tok[tok >= 0]].double() * case["scale"]
        return rows
    if op == "dembed":
        tok = st["tokens"].long()
        there = (tok >= 0).nonzero()[:, 0]
        table = torch.zeros((case["V"], case["d"]), device="cuda", dtype=torch.float64)
        return table.index_put_((tok[there],), st["dy"][there].double() * case["scale"], accumulate=True)
    T, d = case["T"], case["d"]
    parts, sums = [], torch.zeros(d, device="cuda", dtype=torch.float64)
    w = st["w"].double()
    for t0 in range(0, T, max(1, 2 ** 25 // d)):
        r = slice(t0, min(T, t0 + max(1, 2 ** 25 // d)))
        x = st["x"][r].double()
        if op == "dnorm":
            x.requires_grad_(True)
            weight = w.clone().requires_grad_(True)
            y = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * weight
            loss = (y * st["dy"][r].double()).sum()
            if st["res"] is not None:
                loss = loss + (x * st["res"][r].double()).sum()
            dx, dw = torch.autograd.grad(loss, (x, weight))
            sums += dw
            parts.append(dict(dx=dx))
            continue
        o = {}
        if st["res"] is not None:
            o["h"] = (x + st["res"][r].double()).to(st["res"].dtype).double()
            x = o["h"]
        o["rstd"] = 1 / torch.sqrt(x.square().mean(1) + EPS)
        y = x * o["rstd"][:, None] * w
        if case["y"] == "e4m3":
            group = case["group"] or d
            o["scale"] = torch.stack([c.abs().amax(1) for c in y.split(group, 1)], 1) / 448
            o["scale"][o["scale"] == 0] = 1
            wide = o["scale"].repeat_interleave(group, 1)[:, :d]
            o["values"] = _e4m3(y / wide) * wide
        else:
            o["y"] = y
        parts.append(o)
    whole = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    if op == "dnorm":
        whole["dweight"] = sums
    return whole
