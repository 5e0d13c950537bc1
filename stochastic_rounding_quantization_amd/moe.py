"""A mixture-of-experts SwiGLU layer on the library's calls: MXFP4 forward, S3R-EC INT8 backward.

    python -m stochastic_rounding_quantization_amd.moe [--tokens T] [--experts E] [--top-k K] [--width D] [--ff F]

runs one training step (forward and backward) and one decoding step of a layer with random weights and prints
their times.  ``MoeLayer`` is the path itself:

forward   route the logits; the tokens' rows in the experts' order times the experts' gate and up weights (one
          stacked product, 4-bit weights and rows); silu(gate) * up rounded straight into the down product's
          rows; the experts' outputs summed into the tokens with the router's weights.
backward  the sum's gradients; the router's; each projection as the grouped INT8 path takes it (G rounded with
          S3R-EC, dX and dW from one set of codes, up to its 131072 rows); the rows' gradients summed back into the
          tokens.  silu(gate) * up and the joining of the gate and up gradients are torch operations.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

from . import s3r


@dataclass
class Saved:
    """What a backward pass needs of its forward pass."""
    x: object
    logits: object
    routed: s3r.Routed
    gate_up: object        # bf16 [R x 2 F]: the pre-activations, gate columns first
    rows: object           # bf16 [R x D]: the experts' outputs


class _Codes:
    """A weight's codes, kept between the calls that need them and made again when the weight has changed.

    ``of`` sees a change that torch counts (an operation in place) and another tensor; ``renew`` is for the others.
    The same tensor's codes keep their buffers.  A call on another stream than the one that made the codes waits for
    them.  While a graph is recorded, ``of`` makes a changed weight's codes as a part of the graph and keeps nothing.
    """

    def __init__(self, make):
        self.make = make                # make(W, codes or None): the codes of W, in the buffers given
        self.codes = self.weight = self.version = self.stream = self.ready = None

    def of(self, W):
        import torch
        if self.weight is not W or self.version != _version(W):
            if torch.cuda.is_current_stream_capturing():
                return self.make(W, None)
            self.renew(W)
        elif self.stream != s3r._stream(None) and not torch.cuda.is_current_stream_capturing():
            self.ready.wait()           # (torch.cuda.graph synchronises the device before it records)
        return self.codes

    def renew(self, W):
        import torch
        recording = torch.cuda.is_current_stream_capturing()
        if recording and self.weight is not W:
            return                      # no buffers yet that outlive the graph
        self.codes = self.make(W, self.codes if self.weight is W else None)
        self.weight, self.version = W, _version(W)
        if not recording:
            self.stream, self.ready = s3r._stream(None), self.ready or torch.cuda.Event()
            self.ready.record()


def _version(W):
    return None if W.is_inference() else W._version


class MoeLayer:
    """gate_up: bf16 [E x 2F x D] (an expert's gate rows, then its up rows), down: bf16 [E x D x F].

    The layer keeps codes of the weights: MXFP4 from the start, INT8 from the first backward pass.  It follows weights
    that torch's operations change in place, as an optimizer's step does, or that other tensors replace.  After changes
    that torch does not count (through ``.data``, by a kernel that was given the address, by the replay of a graph, to
    inference tensors), and before the replay of a graph that holds the layer's own calls, call ``weights_changed``.
    """

    def __init__(self, gate_up, down, top_k, **router):
        self.gate_up, self.down, self.top_k, self.router = gate_up, down, top_k, router
        self.ff = down.shape[2]
        self._mx = _Codes(_mx_weights), _Codes(_mx_weights)
        self._int8 = _Codes(_int8_gate_up), _Codes(_int8_weights)
        for codes, W in zip(self._mx, (gate_up, down)):
            codes.renew(W)

    @property
    def mx_gate_up(self):
        return self._mx[0].of(self.gate_up)

    @property
    def mx_down(self):
        return self._mx[1].of(self.down)

    def weights_changed(self):
        """Make the codes that the layer keeps again, in their buffers, from the weights as they are."""
        for pair in (self._mx, self._int8):
            for codes, W in zip(pair, (self.gate_up, self.down)):
                if codes.weight is not None:
                    codes.renew(W)

    def forward(self, x, logits, bias=None):
        """(y, Saved) of tokens x [T x D] bf16 with router logits [T x E]."""
        import torch
        r = s3r.route(logits, self.top_k, bias=bias, **self.router)
        a = s3r.mx_linear(x, self.mx_gate_up, offsets=r.offsets, index=r.row_slot, index_div=self.top_k)
        rows = s3r.mx_linear(a[:, :self.ff], self.mx_down, up=a[:, self.ff:], offsets=r.offsets,
                             out_dtype=torch.bfloat16)
        return s3r.combine(rows, r), Saved(x, logits, r, a, rows)

    def backward(self, saved: Saved, dy, *, seed=0, layer_id=0):
        """(dx f32, dlogits, dgate_up f32, ddown f32) from dy [T x D] bf16."""
        import torch
        r, F = saved.routed, self.ff
        if dy.shape[0] == 0:             # the grouped calls take no empty lists of steps
            zeros = dict(dtype=torch.float32, device=dy.device)
            return (torch.zeros(dy.shape, **zeros), torch.empty_like(saved.logits),
                    torch.zeros(self.gate_up.shape, **zeros), torch.zeros(self.down.shape, **zeros))
        gate_w, up_w = self._int8[0].of(self.gate_up)
        down_w = self._int8[1].of(self.down)
        gate, up = saved.gate_up[:, :F].contiguous(), saved.gate_up[:, F:].contiguous()
        drows, dweights = s3r.combine_backward(dy, saved.rows, r)
        dlogits = s3r.route_backward(r, saved.logits, dweights)
        g = gate.float()
        hidden = (g * torch.sigmoid(g) * up.float()).to(torch.bfloat16)
        dh, ddown = _linear_backward(drows, _int8_rows(hidden, r.offsets), down_w, r.offsets, seed, 4 * layer_id)
        dgate, dup = s3r.swiglu_backward(dh, gate, up)
        xq = _int8_rows(s3r.dispatch(saved.x, r), r.offsets)
        dxr, dwg = _linear_backward(dgate, xq, gate_w, r.offsets, seed, 4 * layer_id + 1)
        dxr, dwu = _linear_backward(dup, xq, up_w, r.offsets, seed, 4 * layer_id + 2, into=dxr)
        return s3r.combine(dxr, r, weighted=False), dlogits, torch.cat([dwg, dwu], dim=1), ddown


def _mx_weights(W, codes):
    """MXFP4 rows of W [E x N x K]."""
    if codes is None:
        return s3r.mx_rows(W)
    s3r.s3r_mx_rows(W, codes)
    return codes


def _int8_weights(W, codes):
    """(codes [E x N x K], s_w [E x N], r_W [E x K]) of W [E x N x K]."""
    import torch
    (E, N, K), dev = W.shape, W.device
    d = s3r.qdesc(E * N, K, N, s3r.RTNE, s3r.EC_NONE, s3r.PER_TOKEN)
    Q, s_w, r_W = codes or (s3r.q_buffer(E * N, K, dev).unflatten(0, (E, N)),
                            torch.empty(E, N, dtype=torch.float32, device=dev),
                            torch.empty(E, K, dtype=torch.int32, device=dev))
    ws = torch.empty(s3r.s3r_quantize_workspace(d), dtype=torch.uint8, device=dev)
    s3r.s3r_quantize(d, W.reshape(E * N, K), None, None, Q.flatten(0, 1), s_w, r_W, ws=ws)
    return Q, s_w, r_W


def _int8_gate_up(W, codes):
    """Those of the gate rows and those of the up rows."""
    F = W.shape[1] // 2
    return [_int8_weights(w, c) for w, c in zip((W[:, :F], W[:, F:]), codes or (None, None))]


def _int8_rows(X, offsets):
    """(codes [R x K], s_x [R], xs [E x K]) of the experts' rows."""
    import torch
    (R, K), E, dev = X.shape, offsets.numel() - 1, X.device
    d = s3r.qdesc(R, K, 1, s3r.RTNE, s3r.EC_NONE, s3r.PER_TOKEN)
    Q, s = s3r.q_buffer(R, K, dev), torch.empty(R, dtype=torch.float32, device=dev)
    xs = torch.empty(E, K, dtype=torch.int32, device=dev)
    ws = torch.empty(s3r.s3r_grouped_workspace(d, E, K), dtype=torch.uint8, device=dev)
    s3r.s3r_grouped_quantize(d, offsets, X, None, None, Q, s, xs, ws=ws)
    return Q, s, xs


def _linear_backward(G, xq, wq, offsets, seed, layer, into=None):
    """(dX rows f32, dW [E x N x K] f32) of the experts' linear layers; dX is added into ``into``."""
    import torch
    (R, N), E, dev = G.shape, offsets.numel() - 1, G.device
    (Xq, s_x, xs), (Wq, s_w, r_W) = xq, wq
    K = Xq.shape[1]
    f32 = dict(dtype=torch.float32, device=dev)
    d = s3r.qdesc(R, N, 1, s3r.S3R, s3r.EC_TWO_WAY, s3r.PER_TENSOR, layer, seed)
    Q, delta = s3r.q_buffer(R, N, dev), torch.empty(E, **f32)
    ec = torch.empty(R, **f32), torch.empty(E, N, **f32), torch.empty(E, **f32)
    ws = torch.empty(s3r.s3r_grouped_workspace(d, E, K), dtype=torch.uint8, device=dev)
    s3r.s3r_grouped_quantize(d, offsets, G, s_x, s_w, Q, delta, None, *ec, ws=ws)
    dX = torch.empty(R, K, **f32) if into is None else into
    s3r.s3r_grouped_backward_dx(d, offsets, Q, delta, Wq, s_x, r_W, *ec, dX, ws=ws, accumulate=into is not None)
    dW = torch.empty(E, N, K, **f32)
    s3r.s3r_grouped_backward_dw(d, offsets, Q, delta, Xq, s_w, xs, *ec, dW, ws=ws)
    return dX, dW


def main(argv=None) -> None:
    import torch
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 16384), ("experts", 64), ("top-k", 2), ("width", 2048), ("ff", 1408), ("steps", 5)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    g = torch.Generator("cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    layer = MoeLayer(normal(a.experts, 2 * a.ff, a.width, std=0.02), normal(a.experts, a.width, a.ff, std=0.02), a.top_k)
    x, logits, dy = normal(a.tokens, a.width), normal(a.tokens, a.experts), normal(a.tokens, a.width, std=1e-4)

    def train():
        y, saved = layer.forward(x, logits)
        return layer.backward(saved, dy)

    for what, step in (("training step", train), ("decoding step, 16 tokens", lambda: layer.forward(x[:16], logits[:16]))):
        step()
        torch.cuda.synchronize()
        t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0.record()
        for _ in range(a.steps):
            step()
        t1.record()
        torch.cuda.synchronize()
        print(f"{what}: {t0.elapsed_time(t1) / a.steps:.3f} ms", flush=True)


if __name__ == "__main__":
    main()
