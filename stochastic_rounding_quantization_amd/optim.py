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

    bf16 weights are rounded to nearest after each step, so steps that are small beside 2^-9 of a weight are lost in part: of
    lr 0.02 on weights of 0.02 (1408 x 2048) all arrives, with an error of 0.08 of the step by rounding, of lr 0.001 only 0.56.
    Where steps are so small, keep the weights in f32, update those, and copy them into the layer's bf16 tensors after each step.
    """

    def __init__(self, weights, lr, *, momentum=0.95, nesterov=True, decay=0.0, steps=5, coeffs=s3r.NS_COEFFS, eps=1e-7):
        import torch
        self.weights, self.lr, self.momentum, self.nesterov, self.decay = list(weights), lr, momentum, nesterov, decay
        self.steps, self.coeffs, self.eps = steps, coeffs, eps
        self._workspaces()
        self.buffers = [torch.zeros(W.shape, dtype=torch.float32, device=W.device) for W in self.weights]

    def _update(self, W):
        """How W's update is scaled and kept, and the steps: what s3r_orthogonalize is told."""
        N, K = W.shape[-2:]
        return dict(steps=self.steps, coeffs=self.coeffs, eps=self.eps, scale=-self.lr * max(1.0, N / max(K, 1)) ** 0.5,
                    keep=1.0 - self.lr * self.decay)

    def _workspaces(self):
        """The largest workspace of a weight's update; refuses weights and settings that s3r_orthogonalize would refuse."""
        most = 0
        for W in self.weights:
            if W.dim() not in (2, 3):
                raise ValueError("expected weights that are matrices, or several of one size")
            *_, N, K = W.shape
            if W.numel() and (W.stride(-1) != 1 or W.stride(-2) < K or
                              (W.dim() == 3 and W.shape[0] > 1 and W.stride(0) < (N - 1) * W.stride(-2) + K)):
                raise ValueError("expected weights with unit column stride, row after row and matrix after matrix")
            need = s3r.s3r_orthogonalize_workspace(s3r.orth_desc(W.shape, s3r.S3R_F32, s3r._gdtype(W), **self._update(W)))
            if not need:
                raise ValueError("weights or settings out of the update's range")
            most = max(most, need)
        return most

    def step(self, grads):
        """One update from the gradients, in the weights' order (f32 or bf16, of their shapes, any layout).

        What is refused is refused before anything changes, and memory is taken before as well: after an error of these
        kinds the weights and the momentum are as they were.
        """
        import torch
        grads = list(grads)
        if len(grads) != len(self.weights) or any(g.shape != W.shape for g, W in zip(grads, self.weights)):
            raise ValueError("a gradient for every weight, of its shape")
        if not grads:
            return
        most, dev = self._workspaces(), self.weights[0].device
        if any(t.device != dev for t in (*self.weights, *grads, *self.buffers)):
            raise ValueError("tensors on different devices")
        s3r._here(*self.weights)
        with torch.no_grad():
            ws = s3r._scratch(most, dev)
            f32 = [g.dtype is torch.float32 for g in grads]
            scratch = torch.empty(max((W.numel() for W, same in zip(self.weights, f32) if self.nesterov or not same), default=0),
                                  dtype=torch.float32, device=dev)
            for W, g, buf, same in zip(self.weights, grads, self.buffers, f32):
                u = scratch[:W.numel()].view(W.shape) if self.nesterov or not same else buf
                if not same:
                    g = u.copy_(g)
                buf.mul_(self.momentum).add_(g)
                u = torch.add(g, buf, alpha=self.momentum, out=u) if self.nesterov else buf
                s3r.s3r_orthogonalize(u, W, ws=ws, **self._update(W))
                if not W.is_inference():
                    torch.autograd.graph.increment_version(W)
