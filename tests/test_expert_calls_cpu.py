"""Refusals of the routing, expert-row and MXFP4 product calls: every check runs on the host, before any HIP call.

Pointers are invented, aligned addresses: a call that passed its checks would return the architecture's
error here (there is no GPU) or S3R_ERR_HIP, never S3R_OK; each test first shows that its base call gets that far.
"""
import ctypes

import pytest

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


def route(L, ws=P, wsb=1 << 20, logits=P, dtype=0, ld=None, bias=None, ids=P, weights=P, offsets=P, slot_row=P, row_slot=P,
          reserved=0, T=10, E=16, k=2, **kw):
    d = s3r.route_desc(T, E, k, **kw)
    d.reserved = reserved
    return L.s3r_route(ctypes.byref(d), logits, dtype, E if ld is None else ld, bias, ids, weights, offsets, slot_row,
                       row_slot, ws, wsb, None)


@pytest.mark.parametrize("kw, rc", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(E=128, k=65), UNSUPPORTED), (dict(groups=3), INVALID), (dict(groups=0), INVALID),
    (dict(E=130, groups=65), UNSUPPORTED), (dict(groups=4, keep=5), INVALID), (dict(groups=4, keep=0), INVALID),
    (dict(groups=16, keep=1, k=2), INVALID), (dict(groups=16, keep=8, group_top=2), INVALID),
    (dict(group_top=3), UNSUPPORTED), (dict(group_top=0), UNSUPPORTED), (dict(score=2), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(reserved=1), INVALID),
    (dict(T=1 << 31), INVALID), (dict(T=1 << 30, k=2), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(ld=15), INVALID),
    (dict(logits=None), INVALID), (dict(logits=P + 2), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(offsets=None), INVALID), (dict(offsets=P + 4), INVALID), (dict(slot_row=None), INVALID),
    (dict(row_slot=None), INVALID), (dict(row_slot=P + 2), INVALID), (dict(bias=P + 1), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 128), INVALID), (dict(wsb=256), WORKSPACE)])
def test_route_refuses(L, kw, rc):
    assert route(L) in PAST
    assert route(L, **kw) == rc


def test_route_takes_no_tokens_and_its_limits(L):
    assert route(L, T=0, logits=None, ids=None, weights=None, slot_row=None, row_slot=None) in PAST
    assert route(L, E=1024, k=64, groups=64, keep=64, group_top=2) in PAST
    assert L.s3r_route(None, P, 0, 16, None, P, P, P, P, P, P, 1 << 20, None) == INVALID
    assert s3r.s3r_route_workspace(s3r.route_desc(4, 0, 1)) == 0


@pytest.mark.parametrize("kw, rc", [
    (dict(dtype=3), UNSUPPORTED), (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(dw=None), INVALID),
    (dict(dl=None), INVALID), (dict(ld_d=15), INVALID), (dict(ld=3), INVALID), (dict(dl=P + 1), INVALID),
    (dict(dw=P + 2), INVALID)])
def test_route_backward_refuses(L, kw, rc):
    def call(logits=P, dtype=1, ld=16, ids=P, dw=P, dl=P, ld_d=16):
        d = s3r.route_desc(10, 16, 2)
        return L.s3r_route_backward(ctypes.byref(d), logits, dtype, ld, ids, dw, dl, ld_d, None)
    assert call() in PAST
    assert call(**kw) == rc


@pytest.mark.parametrize("kw, rc", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(R=-1), INVALID), (dict(D=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(ld_t=7), INVALID), (dict(ld_r=7), INVALID), (dict(tok=None), INVALID), (dict(rows=None), INVALID),
    (dict(slot_row=None), INVALID), (dict(slot_row=P + 1), INVALID), (dict(tok=P + 1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(T=1 << 30, k=2), INVALID)])
def test_row_moves_refuse(L, kw, rc):
    def calls(T=4, k=2, R=8, D=8, dtype=1, tok=P, ld_t=8, rows=P, ld_r=8, slot_row=P, w=P, dw=P, drows=P):
        return (L.s3r_dispatch(T, k, R, D, dtype, tok, ld_t, slot_row, rows, ld_r, None),
                L.s3r_combine(T, k, R, D, dtype, rows, ld_r, slot_row, w, tok, ld_t, None),
                L.s3r_combine_backward(T, k, R, D, dtype, tok, ld_t, rows, slot_row, w, drows, ld_r, dw, None))
    assert all(c in PAST for c in calls())
    assert all(c in PAST for c in calls(T=0, tok=None, rows=None, slot_row=None, w=None, dw=None, drows=None))
    assert calls(**kw) == (rc, rc, rc)
    assert calls(w=None)[2] == INVALID and calls(dw=None)[2] == INVALID and calls(drows=None)[2] == INVALID
    assert calls(w=None)[1] in PAST and calls(w=P + 2)[1] == INVALID


ROWS, K, STEPS = 300, 200, 2
LD = STEPS * 16384


@pytest.mark.parametrize("kw, rc", [
    (dict(groups=0), INVALID), (dict(groups=4097), INVALID), (dict(rows=-1), INVALID), (dict(K=1 << 24), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(ld=199), INVALID), (dict(A=None), INVALID), (dict(up=P + 1), INVALID),
    (dict(a_rows=299), INVALID), (dict(index=P, div=0), INVALID), (dict(index=P, a_rows=-1), INVALID),
    (dict(index=P, groups=2), UNSUPPORTED), (dict(codes=None), INVALID), (dict(codes=P + 8), INVALID),
    (dict(ld_c=16384), INVALID), (dict(ld_c=LD + 64), INVALID), (dict(scales=None), INVALID), (dict(ld_s=1196), INVALID),
    (dict(ld_s=1201), INVALID), (dict(groups=2, a_stride=299 * 200), INVALID), (dict(groups=2, c_stride=LD), INVALID),
    (dict(groups=2, s_stride=1200), INVALID)])
def test_mx_rows_refuses(L, kw, rc):
    def call(groups=1, rows=ROWS, K=K, A=P, up=None, dtype=1, ld=200, a_stride=60000, a_rows=ROWS, index=None, div=1, codes=P,
             ld_c=LD, c_stride=2 * LD, scales=P, ld_s=1200, s_stride=2400):
        return L.s3r_mx_rows(groups, rows, K, A, up, dtype, ld, a_stride, a_rows, index, div, codes, ld_c, c_stride,
                             scales, ld_s, s_stride, None, None)
    assert call() in PAST and call(groups=2) in PAST and call(index=P, a_rows=5) in PAST
    assert call(rows=0, a_rows=0, A=None, codes=None, scales=None) in PAST
    assert call(**kw) == rc


def pdesc(rows=10, cols=ROWS, depth=K, groups=0, ld_b=LD, ld_bs=1200, b_stride=2 * LD, bs_stride=2400, out=0, reserved=0):
    return s3r.MxPDesc(rows, cols, depth, groups, ld_b, ld_bs, b_stride, bs_stride, out, reserved)


@pytest.mark.parametrize("kw, rc", [
    (dict(rows=-1), INVALID), (dict(cols=1 << 24), INVALID), (dict(depth=-1), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=4097, offsets=P), INVALID), (dict(groups=2), INVALID), (dict(offsets=P), INVALID),
    (dict(groups=2, offsets=P + 4), INVALID), (dict(out=2), UNSUPPORTED), (dict(reserved=1), INVALID),
    (dict(ld_b=16384), INVALID), (dict(ld_bs=1199), INVALID), (dict(groups=2, offsets=P, b_stride=LD), INVALID),
    (dict(groups=2, offsets=P, bs_stride=1200), INVALID), (dict(B=None), INVALID), (dict(Bs=P + 2), INVALID),
    (dict(y=None), INVALID), (dict(y=P + 2), INVALID), (dict(ld_out=299), INVALID), (dict(ld_out=1 << 22), INVALID)])
def test_products_refuse(L, kw, rc):
    def calls(offsets=None, B=P, Bs=P, y=P, ld_out=ROWS, ws=P, wsb=1 << 20, index=None, a_rows=10, A=P, **d):
        d = ctypes.byref(pdesc(**d))
        return (L.s3r_mx_product(d, A, LD, P, 40, offsets, B, Bs, y, ld_out, None, None),
                L.s3r_mx_linear(d, A, None, 1, 200, a_rows, index, 1, offsets, B, Bs, y, ld_out, None, ws, wsb, None))
    assert all(c in PAST for c in calls()) and all(c in PAST for c in calls(groups=2, offsets=P))
    assert calls(**kw) == (rc, rc)
    assert calls(A=None) == (INVALID, INVALID)
    assert calls(wsb=256)[1] == WORKSPACE and calls(ws=None)[1] == INVALID and calls(a_rows=9)[1] == INVALID


def test_product_refuses_operands(L):
    d = ctypes.byref(pdesc())
    assert L.s3r_mx_product(d, P, 16384, P, 40, None, P, P, P, ROWS, None, None) == INVALID
    assert L.s3r_mx_product(d, P, LD, P, 36, None, P, P, P, ROWS, None, None) == INVALID
    assert L.s3r_mx_product(d, P, LD, P + 1, 40, None, P, P, P, ROWS, None, None) == INVALID
    assert L.s3r_mx_product(None, P, LD, P, 40, None, P, P, P, ROWS, None, None) == INVALID
    assert s3r.s3r_mx_linear_workspace(-1, 5) == 0 and s3r.s3r_mx_linear_workspace(0, 0) >= 256
    # codes of all rows have to stay below 2^32 bytes
    d = ctypes.byref(pdesc(rows=(1 << 24) - 1, depth=1 << 20, cols=1, ld_b=8192 * 16384, ld_bs=4))
    assert L.s3r_mx_linear(d, P, None, 1, 1 << 20, (1 << 24) - 1, None, 1, None, P, P, P, 1, None, P, 1 << 40, None) == INVALID


def test_binding_checks_tensors():
    import torch
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    w = s3r.MxRows(torch.zeros(1, 1, 16384, dtype=torch.uint8), torch.zeros(1, 1, 20, dtype=torch.uint8), 5, 8)
    with pytest.raises(ValueError):
        s3r.s3r_combine(f, i.long(), None, f)
    with pytest.raises(ValueError):
        s3r.s3r_combine(f, i, torch.zeros(4, 3), f)
    with pytest.raises(ValueError):
        s3r.s3r_dispatch(f, i, f.bfloat16())
    with pytest.raises(ValueError):
        s3r.s3r_mx_linear(f, w, torch.zeros(4, 6))
    with pytest.raises(ValueError):
        s3r.s3r_mx_linear(f, w, torch.zeros(4, 5), index=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        s3r.s3r_mx_linear(f, w, torch.zeros(4, 5), offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        s3r.s3r_route(s3r.route_desc(4, 8, 2), f, None, i, torch.zeros(4, 2), torch.zeros(8, dtype=torch.int64), i, i.reshape(-1), None)


def test_binding_refuses_short_codes_and_scales(L):
    """An MxRows built by hand, a buffer of fewer rows, steps or matrices than it says: before anything is read."""
    import torch
    A, y = torch.zeros(300, 200), torch.zeros(300, 300)
    off = torch.zeros(3, dtype=torch.int64)
    ws = torch.empty(s3r.s3r_mx_linear_workspace(300, 200) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]

    def calls(m):
        """With m as the result, and as each operand."""
        good = s3r.mx_rows_buffer(300, 200, "cpu")
        both = torch.zeros(2, 300, 200)
        if m.groups == 2:
            return [lambda: s3r.s3r_mx_rows(both, m, stream=0),
                    lambda: s3r.s3r_mx_product(good, m, y, offsets=off, stream=0),
                    lambda: s3r.s3r_mx_linear(A, m, y, offsets=off, ws=ws, stream=0)]
        return [lambda: s3r.s3r_mx_rows(A, m, stream=0), lambda: s3r.s3r_mx_product(m, good, y, stream=0),
                lambda: s3r.s3r_mx_product(good, m, y, stream=0), lambda: s3r.s3r_mx_linear(A, m, y, ws=ws, stream=0)]

    for groups in (1, 2):
        full = s3r.mx_rows_buffer(300, 200, "cpu", groups)
        c, s = full.codes, full.scales
        for codes, scales in ((c[:, :1].contiguous(), s), (c[..., :16384].contiguous(), s), (c[:-1], s), (c.flatten()[1:], s),
                              (c, s[:, :1].contiguous()), (c, s[..., :-4].contiguous()), (c, s[:-1]), (c, s.flatten()[1:]),
                              (torch.empty(*c.shape, 2, dtype=torch.uint8)[..., 0], s)):
            for call in calls(s3r.MxRows(codes, scales, 300, 200, groups)):
                with pytest.raises(ValueError):
                    call()
        for call in calls(s3r.MxRows(torch.cat([c, c]), torch.cat([s, s]), 300, 200, groups)):
            with pytest.raises(s3r.S3RError) as e:       # larger than they need be, they pass, as far as to the missing GPU
                call()
            assert e.value.code in PAST


def test_product_descriptors_follow_the_rows_they_are_for():
    import torch
    w = s3r.mx_rows_buffer(300, 200, "cpu")
    first = s3r._mx_pdesc(4, w, torch.zeros(4, 300), None)
    w.rows = 200
    second = s3r._mx_pdesc(4, w, torch.zeros(4, 200), None)
    assert (first.cols, second.cols, second.ld_bs) == (300, 200, 800)


def test_no_rows_of_a_source_that_has_some(L):
    """An empty index has no address."""
    assert L.s3r_mx_rows(1, 0, K, P, None, 1, 200, 60000, 5, None, 1, None, LD, 2 * LD, None, 0, 0, None, None) in PAST
    d = ctypes.byref(pdesc(rows=0, groups=2))
    assert L.s3r_mx_linear(d, P, None, 1, 200, 5, None, 2, P, P, P, None, ROWS, None, P, 1 << 20, None) in PAST
    assert L.s3r_mx_rows(1, 1, K, P, None, 1, 200, 60000, 5, None, 1, P, LD, 2 * LD, P, 4, 0, None, None) == INVALID
