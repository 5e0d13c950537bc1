"""The INT8 forward product of a linear layer, y = X W^T on the forward quantizer's codes.  (Oracle: test use only.)

S3R page, "Quantized Backpropagation with Stochastic Rounding": the forward operands are rounded RTNE to S8 with
per-token scales s_x and per-output-channel scales s_w (quantize.forward_operand).  The page leaves the product's own
arithmetic open; here y = fl(fl(s_x s_w) fl(acc)) + bias in fp32 with acc the exact integer sum, then bf16 if asked.
"""
from __future__ import annotations

import numpy as np

from . import quantize as oq, swiglu

F = np.float32


def hidden(gate, up):
    """silu(gate) * up in fp32 with the glue's operations, not rounded to bf16."""
    with np.errstate(all="ignore"):
        return (swiglu.silu_parts(gate)[1] * np.asarray(up, F)).astype(F)


def rows(M, up=None):
    """(codes int8 [R x K], steps f32 [R], flags) of the rows of M (f32 values)."""
    M = np.asarray(M, F)
    out = oq.quantize(M if up is None else hidden(M, up), "f32", mode=oq.RTNE, scale=oq.PER_TOKEN)
    return out["Q"], out["delta"], out["flags"]


def product(qa, sa, qb, sb, bias=None, bf16=False):
    """f32 [M x N]: the result, rounded to bf16's values if asked."""
    acc = qa.astype(np.float64) @ qb.astype(np.float64).T              # exact below 2^53
    with np.errstate(all="ignore"):
        y = (np.asarray(sa, F)[:, None] * np.asarray(sb, F)[None, :]) * acc.astype(F)
        if bias is not None:
            y = y + np.asarray(bias, F)
    return swiglu.bf16_to_f32(swiglu.round_bf16(y)) if bf16 else y
