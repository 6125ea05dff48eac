"""Distillation of a 2:4 sparse student from its dense teacher.

A pruned model recovers by learning from the model it was pruned from. What the
student sees of the teacher is a list per token: the teacher's most probable
tokens and their log probabilities, as p24_token_logprobs finds them. DistillHead
holds the student's head (the unembedding): logits, loss and gradients, one pass
over the logits and in place, so that one [M, V] buffer is all it needs.
DistillStep runs a whole step of a student whose last layer is a 2:4 FFN: prune,
forward, head, loss and backward, on the library's calls.

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
            N.prune24_compress_both(W_up, self.up, self.up_T)
            N.prune24_compress_both(W_down, self.down, self.down_T)
            H = N.spmm24_fwd(X, self.up, b_up, relu=True)
            Y = N.spmm24_fwd(H, self.down, b_down)
            o = self.head.step(Y, W_head, top_idx, top_logp, dkl, labels, dce, temperature, tail)
            o["dW_head"] = o.pop("dW")
            dY = o.pop("dY")
            o["db_up"] = torch.empty(ffn, dtype=torch.float32, device=X.device)
            dH = N.spmm24_bwd_dx(dY, self.down_T, gate=H, dbias=o["db_up"])
            o["db_down"] = N.p24_colsum(dY)
            o["dW_down"] = N.masked_dw_gemm(dY, H, self.down)
            o["dX"] = N.spmm24_bwd_dx(dH, self.up_T)
            o["dW_up"] = N.masked_dw_gemm(dH, X, self.up)
        return o
