"""Distillation of a 2:4 sparse student from its dense teacher.

A pruned model recovers by learning from the model it was pruned from. What the
student sees of the teacher is a list per token: the teacher's most probable
tokens and their log probabilities, as p24_token_logprobs finds them. DistillHead
holds the student's head (the unembedding): logits, loss and gradients, one pass
over the logits and in place, so that one [M, V] buffer is all it needs.
DistillStep runs a whole step of a student whose last layer is a 2:4 FFN: prune,
forward, head, loss and backward, on the library's calls. StudentStep runs one from
tokens to clipped gradients: embedding, a pre-norm 2:4 FFN with its residual, a norm
in front of the head, and the backward of all of it.

A call with stream=s is the call under torch.cuda.stream(s): what it allocates, intermediates that
are dropped when it returns among them, is that stream's memory.
"""
from __future__ import annotations

import torch

from . import _native as N


def _shape(t: torch.Tensor | None, shape: tuple, name: str) -> None:
    """The calls below take sizes from their inputs and write that much to this module's buffers."""
    if t is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")


class DistillHead:
    """Logits = Y W^T of M tokens over a vocabulary of V (a multiple of 8), with the loss
    of p24_distill_topk on them."""

    def __init__(self, M: int, d: int, V: int, device="cuda"):
        if V % 8 or d % 8:
            raise ValueError("the head's products need V and d to be multiples of 8")
        bf = torch.bfloat16
        self.M, self.d, self.V = M, d, V
        self.logits = torch.empty((M, V), dtype=bf, device=device)    # and their gradient, in place
        self.W_T = torch.empty((d, V), dtype=bf, device=device)       # for the product with the gradient

    def _product(self, Y: torch.Tensor, W: torch.Tensor) -> None:
        """Logits of hidden states under a head of any width (a teacher's may differ from d)."""
        _shape(Y, (self.M, Y.shape[-1]), "Y")
        _shape(W, (self.V, Y.shape[-1]), "W")
        N.p24_gemm_nt(Y, W, self.logits)

    def teacher_list(self, Y: torch.Tensor, W: torch.Tensor, k: int, temperature: float = 1.0,
                     out: dict | None = None, stream=None) -> dict:
        """A teacher's list for these tokens from its last hidden states Y [M, d] and its head
        W [V, d]: top_idx, top_logp [M, k], and its entropy, all of softmax(logits / temperature).
        Uses this head's logits buffer."""
        with N._on(stream):
            self._product(Y, W)
            return N.p24_token_logprobs(self.logits, k=k, temperature=temperature, out=out)

    def score(self, Y: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, stream=None) -> dict:
        """Log probabilities of tokens (int32 [M]) and the entropy, e.g. of held-out text."""
        with N._on(stream):
            self._product(Y, W)
            return N.p24_token_logprobs(self.logits, tokens)

    def step(self, Y: torch.Tensor, W: torch.Tensor, top_idx: torch.Tensor, top_logp: torch.Tensor, dkl: torch.Tensor,
             labels: torch.Tensor | None = None, dce: torch.Tensor | None = None, temperature: float = 1.0,
             tail: bool = True, out: dict | None = None, stream=None) -> dict:
        """The loss of hidden states Y [M, d] under the head W [V, d], and its gradients: kl (and ce)
        [M], dY [M, d], dW [V, d]. dkl, dce: each token's weight in the loss (fp32 [M]).
        top_logp: the teacher's log probabilities at this temperature, as teacher_list gives them; the
        teacher is renormalised on its list (tail=False) or has the rest as one bucket (tail=True)."""
        given = {} if out is None else out
        _shape(Y, (self.M, self.d), "Y")
        _shape(given.get("dY"), (self.M, self.d), "dY")
        _shape(given.get("dW"), (self.V, self.d), "dW")
        with N._on(stream):
            if not tail and temperature != 1.0:
                # p24_distill_topk divides a list that it renormalises by the temperature: this one is at it
                top_logp = top_logp * temperature
            self._product(Y, W)
            o = N.p24_distill_topk(self.logits, top_idx, top_logp, labels, temperature, tail, dkl, dce,
                                   out={**given, "dlogits": self.logits})
            N.p24_transpose(W, self.W_T)
            o["dY"] = N.p24_gemm_nt(self.logits, self.W_T, given.get("dY"))
            o["dW"] = N.p24_gemm_tn(self.logits, Y, given.get("dW"))
        return o


class DistillStep:
    """One training step of a student Y = FFN(X), logits = Y W_head^T, with a 2:4 FFN (up, ReLU, down;
    fresh masks every step) and double-pruned backward products, against a teacher's list."""

    def __init__(self, M: int, d: int, ffn: int, V: int, device="cuda"):
        self.head = DistillHead(M, d, V, device)
        self.ffn = ffn
        S = N.Sparse24.empty
        self.up, self.up_T = S(ffn, d, device), S(d, ffn, device)
        self.down, self.down_T = S(d, ffn, device), S(ffn, d, device)

    def run(self, X, W_up, b_up, W_down, b_down, W_head, top_idx, top_logp, dkl, labels=None, dce=None,
            temperature: float = 1.0, tail: bool = True, stream=None) -> dict:
        """Returns kl (and ce) per token and the gradients dX, dW_up, db_up, dW_down, db_down, dW_head."""
        M, d, ffn = self.head.M, self.head.d, self.ffn
        for t, shape, name in ((X, (M, d), "X"), (W_up, (ffn, d), "W_up"), (b_up, (ffn,), "b_up"),
                               (W_down, (d, ffn), "W_down"), (b_down, (d,), "b_down"),
                               (W_head, (self.head.V, d), "W_head")):
            _shape(t, shape, name)
        with N._on(stream):
            H, Y = self._forward(X, W_up, b_up, W_down, b_down)
            o = self.head.step(Y, W_head, top_idx, top_logp, dkl, labels, dce, temperature, tail)
            o["dW_head"] = o.pop("dW")
            self._backward(o, o.pop("dY"), X, H)
        return o

    def _forward(self, X, W_up, b_up, W_down, b_down):
        N.prune24_compress_both(W_up, self.up, self.up_T)
        N.prune24_compress_both(W_down, self.down, self.down_T)
        H = N.spmm24_fwd(X, self.up, b_up, relu=True)
        return H, N.spmm24_fwd(H, self.down, b_down)

    def _backward(self, o: dict, dY, X, H) -> None:
        """The FFN's gradients for that of its output, put into o."""
        o["db_up"] = torch.empty(self.ffn, dtype=torch.float32, device=X.device)
        dH = N.spmm24_bwd_dx(dY, self.down_T, gate=H, dbias=o["db_up"])
        o["db_down"] = N.p24_colsum(dY)
        o["dW_down"] = N.masked_dw_gemm(dY, H, self.down)
        o["dX"] = N.spmm24_bwd_dx(dH, self.up_T)
        o["dW_up"] = N.masked_dw_gemm(dH, X, self.up)


class StudentStep:
    """One training step of a student from its tokens, against a teacher's list:

        x = scale E[tokens],  h = x + FFN(norm(x; w_in)),  logits = norm(h; w_out) W_head^T

    with a 2:4 FFN as in DistillStep, and its gradients scaled to a norm of at most max_norm. Weights come in a dict
    (bf16 E [V, d], W_up, W_down, W_head [V, d]; fp32 w_in, w_out [d], b_up, b_down), their gradients go out under
    "d" + their names. Without a W_head the head's weights are E (tied), and E has both gradients; norms and biases
    that are None or not there are left out, and have no gradient."""

    MATRICES = ("E", "W_up", "W_down", "W_head")
    VECTORS = ("w_in", "w_out", "b_up", "b_down")

    def __init__(self, M: int, d: int, ffn: int, V: int, scale: float = 1.0, eps: float = 1e-6, device="cuda"):
        self.layer = DistillStep(M, d, ffn, V, device)
        self.scale, self.eps = scale, eps

    def run(self, tokens, weights: dict, top_idx, top_logp, dkl, labels=None, dce=None, temperature: float = 1.0,
            tail: bool = True, max_norm: float | None = 1.0, stream=None) -> dict:
        """Returns kl (and ce) per token, the gradients, and with max_norm their norm before they were scaled.
        tokens: int32 [M]; one outside 0..V-1 is padding."""
        w, head = {k: weights.get(k) for k in self.MATRICES + self.VECTORS}, self.layer.head
        M, d, ffn, V = head.M, head.d, self.layer.ffn, head.V
        tied = w["W_head"] is None
        _shape(tokens, (M,), "tokens")
        for name, shape in (("E", (V, d)), ("w_in", (d,)), ("W_up", (ffn, d)), ("b_up", (ffn,)), ("W_down", (d, ffn)),
                            ("b_down", (d,)), ("w_out", (d,)), ("W_head", (V, d))):
            _shape(w[name], shape, name)
        for name in self.MATRICES[:3]:
            if w[name] is None:
                raise ValueError(f"a step needs {name}")
        with N._on(stream):
            x = N.p24_embed(tokens, w["E"], self.scale)
            a = N.p24_rmsnorm(x, w["w_in"], eps=self.eps)
            H, Y = self.layer._forward(a["y"], w["W_up"], w["b_up"], w["W_down"], w["b_down"])
            b = N.p24_rmsnorm(Y, w["w_out"], residual=x, eps=self.eps, out={"h": Y})
            o = head.step(b["y"], w["E"] if tied else w["W_head"], top_idx, top_logp, dkl, labels, dce, temperature, tail)
            back = N.p24_rmsnorm_bwd(o.pop("dY"), b["h"], w["w_out"], b["rstd"])
            dh, o["dw_out"] = back["dx"], back.get("dweight")
            self.layer._backward(o, dh, a["y"], H)
            back = N.p24_rmsnorm_bwd(o.pop("dX"), x, w["w_in"], a["rstd"], dres=dh, out={"dx": dh})
            o["dw_in"] = back.get("dweight")
            for name in self.VECTORS:
                if w[name] is None:
                    o.pop("d" + name)
            dW = o.pop("dW")
            if tied:
                o["dE"] = N.p24_embed_bwd(back["dx"], tokens, V, self.scale, dW=dW, accumulate=True)
            else:
                o["dW_head"], o["dE"] = dW, N.p24_embed_bwd(back["dx"], tokens, V, self.scale)
            if max_norm is not None:
                o["norm"] = N.p24_clip_grads([o[k] for k in self.gradients(tied) if k in o], max_norm)
        return o

    @classmethod
    def gradients(cls, tied: bool = False) -> list[str]:
        """The names of run's gradients, where every norm and bias has weights."""
        return ["d" + n for n in cls.MATRICES + cls.VECTORS if not (tied and n == "W_head")]
