"""The cases that the language-model head's operators are measured on, and their plain forms.

Four kinds of pass, each over a matrix of logits [T, V] (T token positions, V vocabulary entries):

  score   log probability of each position's token, entropy, and the k most probable alternatives
  dscore  the gradient of those log probabilities and entropies
  step    distillation from a teacher's top-K list, loss and gradient in one call (with the label's cross entropy)
  kl      its forward alone (validation); dkl its backward alone, from the forward's saved statistics

Logits are bf16 as a bf16 head writes them, or fp32. Vocabulary sizes are generic: 32000, 50257 (odd: rows of bf16
that are not 16-byte aligned) and 131072; token counts are those of the FFN workloads (synth24) and of serving.
"""
import math

import torch

own = False


def listed():
    return [
        # one sequence being decoded: the sampled token's log probability and 20 alternatives; all latency
        dict(name="score_1x32000_k20", op="score", T=1, V=32000, dtype="bf16", k=20, tau=0.7, entropy=True, allowed=0),
        # a serving batch whose head writes fp32 logits
        dict(name="score_48x131072_k8_f32", op="score", T=48, V=131072, dtype="f32", k=8, tau=1.0, entropy=True, allowed=0),
        # constrained decoding: a grammar leaves 12 tokens of each row, fewer than the alternatives asked for
        dict(name="score_16x50257_k20_masked", op="score", T=16, V=50257, dtype="bf16", k=20, tau=1.0, entropy=True, allowed=12),
        # perplexity of a pruned model on held-out text: token log probabilities only
        dict(name="score_4096x50257", op="score", T=4096, V=50257, dtype="bf16", k=0, tau=1.0, entropy=False, allowed=0),
        # the teacher's pass over a training batch: its top 64 and its entropy
        dict(name="score_8192x131072_k64", op="score", T=8192, V=131072, dtype="bf16", k=64, tau=1.0, entropy=True, allowed=0),
        # policy gradient with an entropy bonus
        dict(name="dscore_4096x50257", op="dscore", T=4096, V=50257, dtype="bf16", k=0, tau=1.0, entropy=True, allowed=0),
        # the same without the bonus, on fp32 logits of a ragged batch
        dict(name="dscore_1000x32003_f32", op="dscore", T=1000, V=32003, dtype="f32", k=0, tau=0.9, entropy=False, allowed=0),
        # a short distillation micro-batch, list renormalised, no labels
        dict(name="step_256x32000_k32", op="step", T=256, V=32000, dtype="bf16", k=32, tau=1.0, tail=False, labels=False),
        # the distillation step of a full batch: 64 teacher entries and a bucket for the rest, labels mixed in
        dict(name="step_8192x131072_k64_tail", op="step", T=8192, V=131072, dtype="bf16", k=64, tau=1.0, tail=True, labels=True),
        # softened distillation on fp32 logits: two temperatures in one pass (KL at 2, labels at 1)
        dict(name="step_1023x50257_k20_f32", op="step", T=1023, V=50257, dtype="f32", k=20, tau=2.0, tail=False, labels=True),
        # validation loss of the student
        dict(name="kl_4096x50257_k64_tail", op="kl", T=4096, V=50257, dtype="bf16", k=64, tau=1.0, tail=True, labels=True),
        # the backward of a loss whose weights are known only after it (from the saved statistics)
        dict(name="dkl_2048x131072_k64", op="dkl", T=2048, V=131072, dtype="bf16", k=64, tau=1.0, tail=False, labels=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "score", "dscore", "step", "step", "step", "kl", "dkl"])
    V = rng.choice([32000, 50257, 131072]) if rng.random() < 0.3 else _spread(rng, 1000, 131072)
    T = _spread(rng, 1 if op == "score" else 64, 8192)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        T = min(T, 4096)
    tau = rng.choice([1.0, 1.0, 0.7, 2.0])
    if op in ("score", "dscore"):
        k = rng.choice([0, 1, 5, 20, 64]) if op == "score" else 0
        allowed = rng.choice([3, 12, 200]) if op == "score" and T <= 256 and rng.random() < 0.4 else 0
        return dict(op=op, T=T, V=V, dtype=dtype, k=k, tau=tau, entropy=rng.random() < 0.6, allowed=allowed)
    k = rng.choice([1, 8, 20, 32, 64, rng.randint(2, 128)])
    return dict(op=op, T=T, V=V, dtype=dtype, k=k, tau=tau, tail=rng.random() < 0.5, labels=rng.random() < 0.6)


def work(case):
    T, V, es = case["T"], case["V"], 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    rows = T * V * es
    if op == "score":  # tokens in; logp, statistics, entropy and the alternatives out
        small = T * (4 + 4 + 8 + (4 if case["entropy"] else 0) + 8 * case["k"])
        return {"bytes": rows + small, "flops": (6 if case["entropy"] else 4) * T * V}
    if op == "dscore":
        return {"bytes": 2 * rows + T * (4 + 8 + 4 + (8 if case["entropy"] else 0)), "flops": (7 if case["entropy"] else 5) * T * V}
    two = case["labels"] and case["tau"] != 1.0
    small = T * (8 * case["k"] + 16 + 8 + (12 if case["labels"] else 0))
    if op == "kl":
        return {"bytes": rows + small, "flops": (8 if two else 4) * T * V}
    return {"bytes": 2 * rows + small, "flops": ((16 if two else 8) if op == "step" else (8 if two else 4)) * T * V}


# ------------------------------------------------------------------ inputs
def _spots(T, V, k, g):
    """k distinct columns for each of T rows: an arithmetic progression mod V with a random start and step."""
    a = torch.randint(0, V, (T, 1), generator=g, device="cuda")
    b = torch.randint(1, max(2, V // max(k, 1)), (T, 1), generator=g, device="cuda")
    return (a + b * torch.arange(k, device="cuda")) % V


def _rows(z, tau):
    m = z.amax(1)
    e = ((z - m[:, None]) / tau).exp()
    s = e.sum(1)
    return m, s, e


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)
    T, V, k, tau = case["T"], case["V"], case["k"], case["tau"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    z = torch.randn((T, V), generator=g, device="cuda") * 2.5
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    sure = torch.rand((T, 1), generator=g, device="cuda") * 14  # from unsure to nearly certain
    z.scatter_add_(1, labels[:, None], sure)
    st = dict(case=dict(case), op=case["op"], tau=tau, k=k)
    if case["op"] in ("score", "dscore"):
        if case.get("allowed"):
            keep = _spots(T, V, case["allowed"], g)
            keep[:, 0] = labels
            masked = torch.full_like(z, -math.inf)
            z = masked.scatter_(1, keep, z.gather(1, keep))
        tokens = labels.to(torch.int32)
        if T >= 64:
            tokens[torch.rand(T, generator=g, device="cuda") < 0.05] = -1  # padding
        st.update(z=z.to(dt), tokens=tokens, entropy=case["entropy"])
        if case["op"] == "dscore":
            m, s, e = _rows(st["z"].float(), tau)
            st["stats"] = torch.stack([m, s.log()], 1)
            st["g"] = torch.randn(T, generator=g, device="cuda")
            if case["entropy"]:
                st["H"] = s.log() - (e * ((st["z"].float() - m[:, None]) / tau)).sum(1) / s
                st["h"] = torch.full((T,), 0.01, device="cuda")
            st["out"] = torch.empty_like(st["z"])
        else:
            new = lambda *shape, t=torch.float32: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
            st["out"] = dict(logp=new(T), stats=new(T, 2))
            if case["entropy"]:
                st["out"]["entropy"] = new(T)
            if k:
                st["out"].update(top_logp=new(T, k), top_idx=new(T, k, t=torch.int32))
        return st
    # the teacher's list: falling log probabilities over distinct columns, with some mass left for the rest
    idx = _spots(T, V, k, g)
    fall = torch.rand((T, k), generator=g, device="cuda").mul_(3).sort(1, descending=True).values
    mass = 0.5 + 0.49 * torch.rand((T, 1), generator=g, device="cuda")
    val = torch.log_softmax(fall * 2, 1) + mass.log()
    z.scatter_add_(1, idx, (val + 9).clamp_min(0))  # a student that has learnt part of it
    idx = idx.to(torch.int32)
    short = torch.rand((T, 1), generator=g, device="cuda") < 0.1  # some lists are shorter than K
    idx.masked_fill_(short & (torch.arange(k, device="cuda") >= (k + 1) // 2), -1)
    pad = torch.rand(T, generator=g, device="cuda") < 0.05
    w = torch.where(pad, 0.0, 0.7 / T * torch.ones(T, device="cuda")) * 64
    st.update(z=z.to(dt), idx=idx, val=val, tail=case["tail"], dkl=w, dce=w * 0.4, labels=None)
    if case["labels"]:
        st["labels"] = torch.where(pad, -1, labels).to(torch.int32)
    if case["op"] == "dkl":
        st["stats"] = _student(st, st["z"].float())["stats"]
    st["out"] = dict(kl=torch.empty(T, device="cuda"), stats=torch.empty((T, 4), device="cuda"))
    if case["labels"]:
        st["out"]["ce"] = torch.empty(T, device="cuda")
    st["dz"] = torch.empty_like(st["z"]) if case["op"] in ("step", "dkl") else None
    return st


# ------------------------------------------------------------------ plain forms
def _score(st):
    z, tau = st["z"].float(), st["tau"]
    T, V = z.shape
    m, s, e = _rows(z, tau)
    tok = st["tokens"].long()
    ok = tok >= 0
    zt = z.gather(1, tok.clamp_min(0)[:, None])[:, 0]
    out = dict(logp=torch.where(ok, (zt - m) / tau - s.log(), 0.0), stats=torch.stack([m, s.log()], 1))
    if st["entropy"]:
        out["entropy"] = s.log() - torch.where(e > 0, e * ((z - m[:, None]) / tau), 0.0).sum(1) / s
    if st["k"]:
        # by value, ties to the lower column: one whole number that orders both
        bits = (z + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2 ** 32 + (V - 1 - torch.arange(V, device=z.device))
        top = key.topk(st["k"], 1).values
        at = V - 1 - (top & 0xFFFFFFFF)
        out["top_idx"] = at.to(torch.int32)
        out["top_logp"] = (z.gather(1, at) - m[:, None]) / tau - s.log()[:, None]
    return out


def _dscore(st):
    z, tau, g = st["z"].float(), st["tau"], st["g"]
    x = (z - st["stats"][:, :1]) / tau - st["stats"][:, 1:]
    p = x.exp()
    tok = st["tokens"].long()
    g = torch.where(tok >= 0, g, 0.0)
    d = -g[:, None] * p
    if st["entropy"]:
        d -= st["h"][:, None] * p * (x + st["H"][:, None])
    d.scatter_add_(1, tok.clamp_min(0)[:, None], g[:, None])
    return (d / tau).to(st["z"].dtype)


def _teacher(st):
    on = st["idx"] >= 0
    if st["tail"]:
        q = torch.where(on, st["val"].exp(), 0.0)
        return on, q, (1 - q.sum(1)).clamp_min(0)
    v = torch.where(on, st["val"] / st["tau"], -math.inf)
    e = (v - v.amax(1, keepdim=True)).exp()
    return on, e / e.sum(1, keepdim=True), None


def _student(st, z):
    """m, exponentials and sums of the student's rows at the temperature and (for the labels) at 1."""
    m, s, e = _rows(z, st["tau"])
    at = st["idx"].long().clamp_min(0)
    if st["tail"]:  # absent entries of the list go to a column of their own
        away = torch.where(st["idx"] >= 0, at, z.shape[1])
        rest = torch.cat([e, torch.zeros_like(e[:, :1])], 1).scatter_(1, away, 0.0).sum(1)
    if st["labels"] is not None:
        e1 = e if st["tau"] == 1 else (z - m[:, None]).exp()
        s1 = e1.sum(1)
    zero = torch.zeros_like(m)
    stats = torch.stack([m, s.log(), rest.log() if st["tail"] else zero, s1.log() if st["labels"] is not None else zero], 1)
    return dict(at=at, stats=stats)


def _kl(st, z, stats, at):
    on, q, qr = _teacher(st)
    m, ls, lr, l1 = (c for c in stats.unbind(1))
    lp = (z.gather(1, at) - m[:, None]) / st["tau"] - ls[:, None]
    kl = torch.where(q > 0, q * (q.log() - lp), 0.0).sum(1)
    if st["tail"]:
        kl = kl + torch.where(qr > 0, qr * (qr.log() - (lr - ls)), 0.0)
    out = dict(kl=kl, stats=stats)
    if st["labels"] is not None:
        lab = st["labels"].long()
        out["ce"] = torch.where(lab >= 0, l1 - (z.gather(1, lab.clamp_min(0)[:, None])[:, 0] - m), 0.0)
    return out


def _dkl(st, z, stats, at):
    on, q, qr = _teacher(st)
    m, ls, lr, l1 = (c[:, None] for c in stats.unbind(1))
    tau = st["tau"]
    p = ((z - m) / tau - ls).exp()
    w = st["dkl"][:, None] / tau
    if st["tail"]:
        total = q.sum(1, keepdim=True) + qr[:, None]
        d = w * p * (total - qr[:, None] / (lr - ls).exp())
        listed_ = w * (p.gather(1, at) * total - q)
    else:
        d = w * p
        listed_ = d.gather(1, at) - w * q
    at = torch.where(on, at, z.shape[1])  # absent entries go to a column of their own here too
    d = torch.cat([d, torch.zeros_like(m)], 1).scatter_(1, at, listed_)[:, :-1]
    if st["labels"] is not None:
        lab = st["labels"].long()[:, None]
        c = torch.where(lab >= 0, st["dce"][:, None], 0.0)
        p1 = (z - m - l1).exp()
        d = d + (c * p1).scatter_add(1, lab.clamp_min(0), -c)
    return d.to(st["z"].dtype)


def run(st):
    op = st["op"]
    if own:
        import semi_structured_sparse_prune24_gb300 as P

        if op == "score":
            return P.p24_token_logprobs(st["z"], st["tokens"], k=st["k"], temperature=st["tau"], entropy=st["entropy"], out=st["out"])
        if op == "dscore":
            return P.p24_token_logprobs_bwd(st["z"], st["tokens"], st["stats"], st["g"], entropy=st.get("H"), dentropy=st.get("h"),
                                        temperature=st["tau"], dlogits=st["out"])
        kind = dict(labels=st["labels"], temperature=st["tau"], tail=st["tail"])
        dce = None if st["labels"] is None else st["dce"]
        if op == "kl":
            return P.p24_distill_topk(st["z"], st["idx"], st["val"], **kind, out=st["out"])
        if op == "step":
            return P.p24_distill_topk(st["z"], st["idx"], st["val"], **kind, dkl=st["dkl"], dce=dce, out=dict(st["out"], dlogits=st["dz"]))
        return P.p24_distill_topk_bwd(st["z"], st["idx"], st["val"], st["stats"], dkl=st["dkl"], dce=dce, **kind, dlogits=st["dz"])
    if op == "score":
        return _score(st)
    if op == "dscore":
        return _dscore(st)
    z = st["z"].float()
    if op == "dkl":
        return _dkl(st, z, st["stats"], st["idx"].long().clamp_min(0))
    s = _student(st, z)
    out = _kl(st, z, s["stats"], s["at"])
    if op == "step":
        out["dlogits"] = _dkl(st, z, s["stats"], s["at"])
    return out


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Row blocks in fp64: log_softmax for the values, autograd for the gradients."""
    st = prepare(case, seed)
    z, tau, op = st["z"], st["tau"], st["op"]
    T, V = z.shape
    parts = []
    block = max(1, min(T, (1 << 27) // V))
    for t0 in range(0, T, block):
        r = slice(t0, min(T, t0 + block))
        x = z[r].double().requires_grad_(op not in ("score", "kl"))
        n = torch.arange(x.shape[0], device="cuda")
        lp = torch.log_softmax(x / tau, 1)
        m = x.detach().amax(1)
        ls = torch.logsumexp((x.detach() - m[:, None]) / tau, 1)
        if op in ("score", "dscore"):
            tok = st["tokens"][r].long()
            logp = torch.where(tok >= 0, lp[n, tok.clamp_min(0)], 0.0)
            if op == "score":
                o = dict(logp=logp, stats=torch.stack([m, ls], 1))
                if st["entropy"]:
                    o["entropy"] = torch.special.entr(lp.exp()).sum(1)
                if st["k"]:
                    o["top_logp"] = lp.topk(st["k"], 1).values
            else:
                total = (logp * st["g"][r].double()).sum()
                if st["entropy"]:
                    total = total - ((lp.exp() * lp).sum(1) * st["h"][r].double()).sum()
                o = dict(d=torch.autograd.grad(total, x)[0])
            parts.append(o)
            continue
        idx, val = st["idx"][r].long(), st["val"][r].double()
        on = idx >= 0
        mine = lp.gather(1, idx.clamp_min(0))
        zero = torch.zeros_like(m)
        lr = zero
        if st["tail"]:
            q = torch.where(on, val.exp(), 0.0)
            qr = (1 - q.sum(1)).clamp_min(0)
            off = torch.cat([torch.zeros_like(x), torch.zeros_like(x[:, :1])], 1).detach().scatter_(1, torch.where(on, idx, V), 1.0)[:, :-1]
            other = torch.logsumexp(lp.masked_fill(off > 0, -math.inf), 1)
            lr = other.detach() + ls
            kl = torch.special.entr(q).neg().sum(1) - (q * mine).sum(1) + torch.special.entr(qr).neg() - qr * other
        else:
            q = torch.softmax((val / tau).masked_fill(~on, -math.inf), 1)
            kl = torch.special.entr(q).neg().sum(1) - (q * mine).sum(1)
        o, l1 = dict(kl=kl.detach()), zero
        if st["labels"] is not None:
            lab = st["labels"][r].long()
            ce = torch.where(lab >= 0, -torch.log_softmax(x, 1)[n, lab.clamp_min(0)], 0.0)
            l1 = torch.logsumexp(x.detach() - m[:, None], 1)
            o["ce"] = ce.detach()
        if op in ("step", "dkl"):
            total = (kl * st["dkl"][r].double()).sum()
            if st["labels"] is not None:
                total = total + (ce * st["dce"][r].double()).sum()
            o["dlogits"] = torch.autograd.grad(total, x)[0]
        o["stats"] = torch.stack([m, ls, lr, l1], 1)
        parts.append(o)
    whole = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    if op == "dscore":
        return whole["d"]
    if op == "dkl":
        return whole["dlogits"]
    if op == "score" and st["k"]:
        whole["top_idx"] = None
    return whole
