"""Refusals of the INT8 forward calls (host checks, before any HIP call), and pins of their oracle.

Pointers are invented, aligned addresses: a call that passed its checks would return the architecture's
error here (there is no GPU) or S3R_ERR_HIP, never S3R_OK; each test first shows that its base call gets that far.
"""
import ctypes

import numpy as np
import pytest

from oracle import int8, quantize as oq
from stochastic_rounding_quantization_amd import s3r

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
PAST = (-4, -5)                      # the checks are passed: no gfx950, or no device at all
P = 1 << 20


@pytest.fixture(scope="module")
def L():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the invented pointers are for a machine without a GPU")
    return s3r.lib()


ROWS, K, LD = 300, 200, 208


@pytest.mark.parametrize("kw, rc", [
    (dict(groups=0), INVALID), (dict(groups=4097), INVALID), (dict(rows=-1), INVALID), (dict(K=131073), INVALID),
    (dict(K=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(ld=199), INVALID), (dict(A=None), INVALID), (dict(A=P + 1), INVALID),
    (dict(up=P + 1), INVALID), (dict(a_rows=299), INVALID), (dict(index=P, div=0), INVALID),
    (dict(index=P + 2), INVALID), (dict(index=P, a_rows=-1), INVALID), (dict(index=P, groups=2), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(codes=P + 8), INVALID), (dict(ld_c=200), INVALID), (dict(ld_c=192), INVALID),
    (dict(ld_c=1 << 23), INVALID), (dict(delta=None), INVALID), (dict(delta=P + 2), INVALID),
    (dict(groups=2, a_stride=299 * 200), INVALID), (dict(groups=2, c_stride=299 * LD), INVALID),
    (dict(groups=2, c_stride=300 * LD + 8), INVALID)])
def test_rows_refuse(L, kw, rc):
    def call(groups=1, rows=ROWS, K=K, A=P, up=None, dtype=1, ld=200, a_stride=60000, a_rows=ROWS, index=None, div=1, codes=P,
             ld_c=LD, c_stride=300 * LD, delta=P):
        return L.s3r_int_rows(groups, rows, K, A, up, dtype, ld, a_stride, a_rows, index, div, codes, ld_c, c_stride, delta,
                              None, None)
    assert call() in PAST and call(groups=2) in PAST and call(index=P, a_rows=5) in PAST
    assert call(rows=0, a_rows=0, A=None, codes=None, delta=None) in PAST
    assert call(K=0, A=None, codes=None, ld=0) in PAST
    assert call(**kw) == rc


def pdesc(rows=10, cols=ROWS, depth=K, groups=0, ld_b=LD, b_stride=ROWS * LD, out=0, reserved=0):
    return s3r.IntPDesc(rows, cols, depth, groups, ld_b, b_stride, out, reserved)


@pytest.mark.parametrize("kw, rc", [
    (dict(rows=-1), INVALID), (dict(cols=1 << 31), INVALID), (dict(cols=-1), INVALID), (dict(depth=-1), INVALID),
    (dict(depth=131073, ld_b=131088), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=4097, offsets=P), INVALID), (dict(groups=2), INVALID), (dict(offsets=P), INVALID),
    (dict(groups=2, offsets=P + 4), INVALID), (dict(out=2), UNSUPPORTED), (dict(reserved=1), INVALID),
    (dict(ld_b=200), INVALID), (dict(ld_b=192), INVALID), (dict(ld_b=1 << 23), INVALID),
    (dict(groups=2, offsets=P, b_stride=299 * LD), INVALID), (dict(groups=2, offsets=P, b_stride=ROWS * LD + 8), INVALID),
    (dict(B=None), INVALID), (dict(B=P + 8), INVALID), (dict(sb=None), INVALID), (dict(sb=P + 2), INVALID),
    (dict(bias=P + 1), INVALID), (dict(y=None), INVALID), (dict(y=P + 2), INVALID), (dict(ld_out=299), INVALID)])
def test_products_refuse(L, kw, rc):
    def calls(offsets=None, B=P, sb=P, bias=None, y=P, ld_out=ROWS, ws=P, wsb=1 << 20, index=None, a_rows=10, A=P, sa=P, **d):
        d = ctypes.byref(pdesc(**d))
        return (L.s3r_int_product(d, A, LD, sa, offsets, B, sb, bias, y, ld_out, None, None),
                L.s3r_int_linear(d, A, None, 1, 200, a_rows, index, 1, offsets, B, sb, bias, y, ld_out, None, ws, wsb, None))
    assert all(c in PAST for c in calls()) and all(c in PAST for c in calls(groups=2, offsets=P, bias=P))
    assert calls(**kw) == (rc, rc)
    assert calls(A=None) == (INVALID, INVALID) and calls(sa=None)[0] == INVALID and calls(sa=P + 2)[0] == INVALID
    assert calls(wsb=256)[1] == WORKSPACE and calls(ws=None)[1] == INVALID and calls(ws=P + 128)[1] == INVALID
    assert calls(a_rows=9)[1] == INVALID and calls(A=P + 8)[0] == INVALID


def test_products_take_empty_sizes(L):
    d = ctypes.byref(pdesc(rows=0, groups=2))
    assert L.s3r_int_linear(d, P, None, 1, 200, 5, None, 2, P, P, P, None, None, ROWS, None, P, 1 << 20, None) in PAST
    d = ctypes.byref(pdesc(depth=0, ld_b=0))
    assert L.s3r_int_product(d, None, 0, P, None, None, P, P, P, ROWS, None, None) in PAST
    assert L.s3r_int_product(None, P, LD, P, None, P, P, None, P, ROWS, None, None) == INVALID
    assert s3r.s3r_int_linear_workspace(-1, 5) == 0 and s3r.s3r_int_linear_workspace(0, 0) >= 256


@pytest.mark.parametrize("kw, rc", [
    (dict(groups=0), INVALID), (dict(rows=-1), INVALID), (dict(groups=7), INVALID), (dict(groups=4097, offsets=P), INVALID),
    (dict(offsets=P + 4), INVALID), (dict(Q=None), INVALID), (dict(Q=P + 8), INVALID), (dict(ld=200), INVALID),
    (dict(sums=None), INVALID), (dict(sums=P + 2), INVALID), (dict(K=-1), INVALID)])
def test_column_sums_refuse(L, kw, rc):
    def call(groups=4, offsets=None, rows=ROWS, K=K, Q=P, ld=LD, sums=P):
        return L.s3r_int_colsum(groups, offsets, rows, K, Q, ld, sums, None, None)
    assert call() in PAST and call(groups=7, offsets=P) in PAST and call(rows=0, Q=None) in PAST
    assert call(**kw) == rc


def test_binding_checks_tensors(L):
    import torch
    f, y = torch.zeros(4, 8), torch.zeros(4, 5)
    w = s3r.int_rows_buffer(5, 8, "cpu")
    a = s3r.int_rows_buffer(4, 8, "cpu")
    two = s3r.int_rows_buffer(5, 8, "cpu", 2)
    i64 = dict(dtype=torch.int64)
    short = s3r.IntRows(w.codes[:, :4].contiguous(), w.delta, 5, 8)
    ws = s3r.int_linear_buffer(4, 8, "cpu")
    bad = [lambda: s3r.s3r_int_linear(f, w, torch.zeros(4, 6), ws=ws), lambda: s3r.s3r_int_linear(f, two, y, ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y, index=torch.zeros(3, dtype=torch.int32), ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y, offsets=torch.zeros(3, **i64), ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y, bias=torch.zeros(4), ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y, bias=torch.zeros(5).bfloat16(), ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y, up=f.bfloat16(), ws=ws), lambda: s3r.s3r_int_linear(f, short, y, ws=ws),
           lambda: s3r.s3r_int_linear(f, w, y.half(), ws=ws), lambda: s3r.s3r_int_product(a, short, y),
           lambda: s3r.s3r_int_product(short, w, torch.zeros(5, 5)), lambda: s3r.s3r_int_product(two, w, y),
           lambda: s3r.s3r_int_product(a, s3r.int_rows_buffer(5, 9, "cpu"), y),
           lambda: s3r.s3r_int_rows(f, w), lambda: s3r.s3r_int_rows(f.t(), w), lambda: s3r.s3r_int_rows(f, two),
           lambda: s3r.s3r_int_rows(torch.zeros(5, 8), short), lambda: s3r.s3r_int_rows(torch.zeros(5, 8).half(), w),
           lambda: s3r.s3r_int_colsum(a.Q, torch.zeros(1, 8)), lambda: s3r.s3r_int_colsum(f, torch.zeros(1, 8, dtype=torch.int32)),
           lambda: s3r.s3r_int_colsum(a.Q, torch.zeros(1, 7, dtype=torch.int32)),
           lambda: s3r.s3r_int_colsum(a.Q, torch.zeros(2, 8, dtype=torch.int32), offsets=torch.zeros(4, **i64))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: s3r.s3r_int_linear(f, w, y, stream=0, ws=torch.empty(1 << 12, dtype=torch.uint8)),
                 lambda: s3r.s3r_int_product(a, w, y, stream=0), lambda: s3r.s3r_int_rows(f, a, stream=0)):
        with pytest.raises(s3r.S3RError):                # as far as to the missing GPU, or the workspace's alignment
            call()


def test_oracle_rows_are_the_forward_operand():
    r = np.random.default_rng(1)
    X = (r.normal(size=(20, 70)) * 3).astype(np.float32)
    f = oq.forward_operand(X, "f32")
    q, s, flags = int8.rows(X)
    assert np.array_equal(q, f["Q"]) and np.array_equal(s, f["scale"]) and flags == 0
    g, u = X, np.roll(X, 1)
    np.testing.assert_allclose(int8.hidden(g, u), g / (1 + np.exp(-g.astype(np.float64))) * u, rtol=1e-6, atol=1e-9)


def test_oracle_product_against_float64():
    r = np.random.default_rng(2)
    X, W, b = (r.normal(size=s).astype(np.float32) for s in ((9, 300), (7, 300), (7,)))
    (qx, sx, _), (qw, sw, _) = int8.rows(X), int8.rows(W)
    y = int8.product(qx, sx, qw, sw, b)
    exp = (qx * sx[:, None].astype(np.float64)) @ (qw * sw[:, None].astype(np.float64)).T + b
    # three roundings of the product (steps, sum, both) and one of the whole
    assert (np.abs(y - exp) <= 2.0 ** -24 * (3 * np.abs(exp - b) + np.abs(exp)) * (1 + 1e-6)).all()
    # and the codes' values lie within half a step of the inputs'
    full = X.astype(np.float64) @ W.astype(np.float64).T + b
    most = (np.abs(X) + sx[:, None]) @ np.full((300, 7), 0.5) * sw + 0.5 * sx[:, None] * np.abs(W).sum(1)
    assert (np.abs(y - full) <= most).all()
    z = int8.product(qx, sx, qw, sw, b, bf16=True)
    assert (np.abs(z - y) <= 2.0 ** -8 * np.abs(y)).all() and not (z.view(np.uint32) & 0xFFFF).any()
