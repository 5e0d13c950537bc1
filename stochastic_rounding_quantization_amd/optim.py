"""The update of a linear layer's weights from their gradients: momentum, orthogonalised by Newton-Schulz steps.

The S3R page leaves the optimizer open.  ``Muon`` takes the dW of the backward calls (f32) to the weights in one library
call each, s3r_orthogonalize, whose last product writes W = (1 - lr decay) W - lr scale X itself.
"""
from __future__ import annotations

from . import s3r


class Muon:
    """weights: matrices [N x K], or one per expert [E x N x K], f32 or bf16, rows with unit column stride (a stacked
    projection's parts are weights of their own: give its slices).

    step   buf <- momentum buf + dW,  u = dW + momentum buf (Nesterov) or buf,  X = u orthogonalised,
           W <- (1 - lr decay) W - lr sqrt(max(1, N / K)) X, rounded once for bf16 weights.
    The momentum is kept in f32.  torch sees the weights change, as after an operation in place.
    """

    def __init__(self, weights, lr, *, momentum=0.95, nesterov=True, decay=0.0, steps=5, coeffs=s3r.NS_COEFFS, eps=1e-7):
        import torch
        self.weights, self.lr, self.momentum, self.nesterov, self.decay = list(weights), lr, momentum, nesterov, decay
        self.steps, self.coeffs, self.eps = steps, coeffs, eps
        self.buffers = [torch.zeros(W.shape, dtype=torch.float32, device=W.device) for W in self.weights]

    def step(self, grads):
        """One update from the gradients, in the weights' order (f32 or bf16, of their shapes)."""
        import torch
        grads = list(grads)
        if len(grads) != len(self.weights) or any(g.shape != W.shape for g, W in zip(grads, self.weights)):
            raise ValueError("a gradient for every weight, of its shape")
        with torch.no_grad():
            for W, g, buf in zip(self.weights, grads, self.buffers):
                g = g.float()
                buf.mul_(self.momentum).add_(g)
                u = g.add(buf, alpha=self.momentum) if self.nesterov else buf
                N, K = W.shape[-2:]
                s3r.s3r_orthogonalize(u, W, steps=self.steps, coeffs=self.coeffs, eps=self.eps,
                                      scale=-self.lr * max(1.0, N / max(K, 1)) ** 0.5, keep=1.0 - self.lr * self.decay,
                                      ws=s3r.orthogonalize_buffer(W))
                if not W.is_inference():
                    torch.autograd.graph.increment_version(W)
