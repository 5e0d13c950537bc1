"""Routing, its gradient and the experts' row moves on an MI355X against oracle/route.py (float64).

Choices and orders are equal.  Tolerances, from half an ulp U = 2^-24 of fp32 per operation: a softmax
weight exp(x - m) / sum carries |x - m| U through the exponential and at most 64 further roundings; its
gradient twice that on the scale of the largest incoming gradient.  A bf16 result adds half a step of its own, 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import route as ref
from stochastic_rounding_quantization_amd import s3r
from tests._gpu import DEV, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def logits(T, E, dtype, seed=0, ties=False):
    x = np.random.default_rng(seed).normal(size=(T, E)) * 2
    if ties:
        x = np.round(x * 2) / 2
    return torch.from_numpy(x).to(DEV, dtype)


def check(x, top_k, *, score=0, bias=None, renorm=True, scale=1.0, **groups):
    r = s3r.route(x, top_k, score=score, bias=bias, renorm=renorm, scale=scale, **groups)
    torch.cuda.synchronize()
    xs = host(x.double())
    b = None if bias is None else host(bias)
    ids = ref.choose(xs, top_k, score=score, bias=b, **groups)
    np.testing.assert_array_equal(host(r.ids), ids)
    w = ref.weights(xs, ids, score=score, renorm=renorm, scale=scale)
    fine = xs[np.isfinite(xs)]
    span = np.ptp(fine) if fine.size else 0.0
    np.testing.assert_allclose(host(r.weights), w, rtol=U * (64 + 2 * span + 2), atol=1e-37)
    for got, exp in zip((r.offsets, r.slot_row, r.row_slot), ref.order(ids, x.shape[1])):
        np.testing.assert_array_equal(host(got), exp)
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 64, 2), (16, 64, 2), (3, 5, 5), (100, 160, 6), (257, 256, 8),
                                     (700, 60, 4), (40, 1024, 64), (1300, 33, 3), (513, 7, 1)])
def test_route(T, E, k, score, dtype):
    check(logits(T, E, dtype, T + E), k, score=score, renorm=(T + k) % 2 == 0, scale=1.5)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E, k, groups, keep, top", [(256, 8, 8, 4, 2), (60, 4, 3, 2, 1), (160, 6, 5, 1, 2), (64, 3, 64, 3, 1),
                                                     (96, 2, 2, 2, 2)])
def test_route_groups_and_bias(E, k, groups, keep, top, bias, score):
    b = torch.randn(E, device=DEV, generator=torch.Generator(DEV).manual_seed(1)) * 0.1 if bias else None
    check(logits(300, E, torch.float32, E + k), k, score=score, bias=b, groups=groups, keep=keep, group_top=top)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups, keep, top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_infinite_bias(groups, keep, top, score):
    """Experts that a bias of inf puts first tie, to the lower index; -inf puts them last."""
    b = torch.zeros(64, device=DEV)
    b[[3, 8, 20]] = float("inf")
    b[[0, 9, 40]] = float("-inf")
    check(logits(300, 64, torch.float32, 3), 5, score=score, bias=b, groups=groups, keep=keep, group_top=top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_route_of_every_width(dtype, offset):
    """Row ends at every place of a 16-byte word, with +inf around the rows; nothing else of the gradient is written."""
    T = 9
    for E in [*range(1, 34), 127, 129, 131, 252, 255, 257, 1019]:
        k = min(E, 3)
        wide = torch.full((T + 2, E + 21), float("inf"), dtype=dtype, device=DEV)
        x = wide[1:T + 1, offset:offset + E]
        x.copy_(logits(T, E, dtype, E))
        bias = torch.randn(E, device=DEV) * 0.1
        check(x, k, renorm=False)
        r = check(x, k, score=E % 2, bias=bias)
        dw = torch.randn(T, k, device=DEV)
        for score, renorm in ((0, False), (1, False)):
            out = torch.full((T + 2, E + 21), 9.0, dtype=dtype, device=DEV)
            dx = out[1:T + 1, offset:offset + E]
            s3r.s3r_route_backward(s3r.route_desc(T, E, k, score=score, renorm=renorm), x, r.ids, dw, dx)
            xs = host(x.double())
            exp = ref.backward(xs, host(r.ids), host(dw), score=score, renorm=renorm)
            # of a gradient of at most |dw|: exponentials and sums, |x| U and 80 roundings; half a bf16 step
            tol = U * (80 + 4 * np.abs(xs).max()) * np.abs(host(dw)).max() * 4
            step = half(dtype) * (1 + 1e-3) if dtype == torch.bfloat16 else 0.0
            assert (np.abs(host(dx.double()) - exp) <= tol + step * np.abs(exp)).all()
            assert (out == 9).sum() >= out.numel() - dx.numel()


@pytest.mark.parametrize("groups, keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lower_index(groups, keep, bias):
    b = torch.zeros(64, device=DEV) if bias else None
    check(logits(500, 64, torch.bfloat16, 3, ties=True), 6, score=1, bias=b, groups=groups, keep=keep)
    check(torch.zeros(70, 64, device=DEV), 5, bias=b, groups=groups, keep=keep)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_both_zeros_are_one_key(dtype):
    x = torch.where(torch.rand(300, 64, device=DEV, generator=torch.Generator(DEV).manual_seed(4)) < 0.5, -0.0, 0.0)
    x[:, ::5] = -1.0
    for kw in ({}, dict(score=1), dict(groups=4, keep=2), dict(bias=torch.zeros(64, device=DEV))):
        check(x.to(dtype), 6, **kw)


def test_keys_that_only_64_bits_tell_apart():
    # sigmoid(x) + bias of neighbours differ by 2^-30: equal in fp32
    x = torch.zeros(200, 40, device=DEV)
    bias = torch.zeros(40, device=DEV)
    bias[7], bias[30], bias[31] = 2.0 ** -30, 2.0 ** -29, -(2.0 ** -30)
    r = check(x, 4, score=1, bias=bias)
    assert host(r.ids)[0].tolist() == [30, 7, 0, 1]
    check(x, 40, score=0, bias=bias)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_logits(score, renorm):
    x = logits(90, 24, torch.float32, 5)
    m = torch.rand(90, 24, device=DEV, generator=torch.Generator(DEV).manual_seed(2)) < 0.8
    x[m] = float("-inf")
    x[3] = float("-inf")                                     # nothing left
    x[4] = torch.finfo(torch.float32).min                    # the type's lowest value: not masked, all equal
    for kw in ({}, dict(groups=4, keep=2)):
        r = check(x, 5, score=score, renorm=renorm, **kw)
        assert (host(r.weights)[3] == 0).all()


def test_not_a_number_and_infinity():
    x = logits(6, 16, torch.float32, 6)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    for score in (0, 1):
        for renorm in (True, False):
            r = s3r.route(x, 4, score=score, renorm=renorm)
            ids = ref.choose(host(x), 4, score=score)
            np.testing.assert_array_equal(host(r.ids), ids)
            w = host(r.weights)
            assert np.isfinite(w[[0, 3, 4, 5]]).all()
            assert np.isnan(w[1:3]).all() if score == 0 else np.isfinite(w[1:3]).all()


def test_tiny_sigmoid_scores_renormalise():
    x = logits(20, 12, torch.float32, 7) - 150.0             # every score underflows fp32
    r = check(x, 3, score=1)
    np.testing.assert_allclose(host(r.weights).sum(axis=1), 1.0, rtol=8 * U)


def test_sigmoid_scores_of_all_sizes_renormalise():
    """Chosen scores that underflow fp32 beside ones that nearly do, and beside ordinary, masked and NaN ones."""
    check(logits(300, 12, torch.float32, 8) * 25, 12, score=1)
    x = torch.tensor([[-89.0, -51.5, -300, -300], [-59.0, -91, -300, -300], [-87.0, -88, -89, -90], [-104.0, -105, -120, -90],
                      [-300.0, -301, -302, -310], [5.0, -100, -200, 3]], device=DEV)
    for k in (2, 4):
        check(x, k, score=1)
    ninf = float("-inf")
    x = torch.tensor([[ninf, -95.0, ninf, -93], [ninf] * 4, [-95.0, ninf, float("nan"), ninf]], device=DEV)
    r = s3r.route(x, 4, score=1)
    w = host(r.weights)
    assert host(r.ids)[0].tolist() == [3, 1, 0, 2] and (w[1] == 0).all() and np.isnan(w[2]).all()
    np.testing.assert_allclose(w[0], [1 / (1 + np.exp(-2)), 1 / (1 + np.exp(2)), 0, 0], rtol=U * 400)


def test_no_tokens():
    r = s3r.route(torch.empty(0, 8, device=DEV), 2)
    assert host(r.offsets).tolist() == [0] * 9
    assert s3r.route_backward(r, torch.empty(0, 8, device=DEV), torch.empty(0, 2, device=DEV)).shape == (0, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    wide = logits(130, 80, dtype, 8)
    for x in (wide[:, 3:67], wide[:, 8:72], wide[::2, :64]):
        r = check(x, 3)
        d = torch.full((x.shape[0], 70), 7.0, dtype=dtype, device=DEV)
        g = torch.randn(x.shape[0], 3, device=DEV)
        s3r.s3r_route_backward(r.desc, x, r.ids, g, d[:, 5:69])
        same = s3r.route_backward(r, x.contiguous(), g)
        assert torch.equal(d[:, 5:69], same) and (d[:, :5] == 7).all() and (d[:, 69:] == 7).all()


def test_many_tokens_and_one_expert_taking_all():
    x = logits(30000, 64, torch.bfloat16, 9)
    x[:, 17] = 50.0
    r = s3r.route(x, 2)
    ids = host(r.ids)
    assert (ids[:, 0] == 17).all()
    row_slot = np.argsort(ids.reshape(-1), kind="stable")
    np.testing.assert_array_equal(host(r.row_slot), row_slot)
    np.testing.assert_array_equal(host(r.offsets), np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=64))]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 64, 2), (77, 160, 6), (300, 64, 2), (5, 1024, 64), (130, 9, 9), (33, 250, 8)])
def test_route_backward(T, E, k, score, renorm, dtype):
    x = logits(T, E, dtype, T * E)
    r = s3r.route(x, k, score=score, renorm=renorm, scale=1.5)
    g = torch.randn(T, k, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    got = host(s3r.route_backward(r, x, g).double())
    exp = ref.backward(host(x.double()), host(r.ids), host(g), score=score, renorm=renorm, scale=1.5)
    span = np.ptp(host(x.double()))
    tol = 2 * U * (64 + 2 * span) * 1.5 * np.abs(host(g)).max() + (2.0 ** -8 if dtype == torch.bfloat16 else 0) * np.abs(exp)
    assert (np.abs(got - exp) <= tol).all()


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masked_and_foreign_ids(score, renorm):
    x = logits(40, 20, torch.float32, 11)
    x[5] = float("-inf")
    x[6, 3:] = float("-inf")
    x[7] -= 150.0
    r = s3r.route(x, 5, score=score, renorm=renorm)
    r.ids[9, 2], r.ids[10, 0] = -1, 20
    g = torch.randn(40, 5, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    got = host(s3r.route_backward(r, x, g))
    exp = ref.backward(host(x), host(r.ids), host(g), score=score, renorm=renorm)
    assert np.isfinite(got).all() and (got[5] == 0).all()
    assert (np.abs(got - exp) <= 2 * U * (64 + 2 * 160) * np.abs(host(g)).max()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_of_nan_and_infinity(score, renorm, dtype):
    """NaN where the weights of a chosen logit are, and nowhere else."""
    x = logits(40, 20, dtype, 14)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3, :9] = float("-inf")
    x[4, 2], x[4, 7] = float("inf"), float("-inf")
    x[5] = float("nan")
    ids = torch.tensor([[3, 5, 2, 7, 0]] * 40, dtype=torch.int32, device=DEV)
    g = torch.randn(40, 5, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    d = torch.empty_like(x)
    s3r.s3r_route_backward(s3r.route_desc(40, 20, 5, score=score, renorm=renorm), x, ids, g, d)
    got = host(d.double())
    with np.errstate(all="ignore"):
        exp = ref.backward(host(x.double()), host(ids), host(g), score=score, renorm=renorm)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(exp))
    fine = np.isfinite(exp)
    tol = 2 * U * (64 + 2 * 20) * np.abs(host(g)).max() + (half(dtype) if dtype == torch.bfloat16 else 0) * (1 + 1e-3) * np.abs(exp)
    assert (np.abs(got - exp)[fine] <= tol[fine]).all()


# ------------------------------------------------- groups by sums of two ----

SUMS = [(8, 4), (32, 4), (36, 3), (256, 8)]      # experts and groups: of two, of a lane, of neither, of several lanes


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E, groups", SUMS)
@pytest.mark.parametrize("size", [256.0, 2.0 ** 20])
def test_group_sums_that_cancel(E, groups, size, score):
    """A group's two largest keys of opposite signs: their sum is far more exact in fp64 than the keys are in fp32."""
    per = E // groups
    b = torch.full((E,), -size, device=DEV)
    b[::per] = size
    x = logits(4000, E, torch.float32, E)
    check(x, 2, score=score, bias=b, groups=groups, keep=groups // 2, group_top=2)
    check(x, 1, score=score, bias=b, groups=groups, keep=1, group_top=2)          # one key of that size


@pytest.mark.parametrize("E, groups", SUMS)
def test_group_sums_that_only_64_bits_tell_apart(E, groups):
    """Sums of two that differ by 2^-30 around 1, and sums that overflow fp32."""
    per = E // groups
    x = torch.zeros(100, E, device=DEV)
    b = torch.full((E,), -0.25, device=DEV)
    for g in range(groups):
        b[g * per] = ((g * 5 + 3) % groups) * 2.0 ** -30
        b[g * per + 1] = -(2.0 ** -31)
    check(x, 2, score=1, bias=b, groups=groups, keep=1, group_top=2)
    check(x, 3, score=1, bias=b, groups=groups, keep=2, group_top=2)
    for sign in (1.0, -1.0):
        b = torch.full((E,), -3.4e38, device=DEV)
        for g in range(groups):
            b[g * per:g * per + 2] = sign * (2e38 + 1e37 * ((g * 5 + 3) % groups))
            b[g * per + 1] -= 1e36
        check(x, 1, score=1, bias=b, groups=groups, keep=1, group_top=2)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E, groups", SUMS)
def test_group_sums_of_infinities(E, groups, score):
    """inf - inf is no sum: the group ranks last, and no group more than `keep` stays."""
    per = E // groups
    x = logits(300, E, torch.float32, E)
    b = torch.zeros(E, device=DEV)
    b[:per] = float("-inf")
    b[0] = float("inf")
    for keep in (1, 2):
        check(x, 2, score=score, bias=b, groups=groups, keep=keep, group_top=2)
    b[:] = 0
    b[per] = float("inf")                                 # beside masked logits
    x[:150, per + 1:2 * per] = float("-inf")
    x[:20, 2 * per:] = float("-inf")
    x[:10] = float("-inf")
    for keep in (1, 2):
        check(x, 2, score=score, bias=b, groups=groups, keep=keep, group_top=2)


def test_groups_of_two_choose_by_logits_where_scores_meet():
    x = torch.tensor([[40.0, 50.0, 0.0, 0.0], [40.0, 50.0, 60.0, 39.0]], device=DEV)
    r = check(x, 1, score=1, groups=2, keep=1, group_top=2)
    assert host(r.ids).tolist() == [[1], [1]]
    x = torch.tensor([[-800.0, -790.0, 0.0, -1000.0]], device=DEV)
    assert host(check(x, 4, groups=2, keep=2, group_top=2).ids).tolist() == [[2, 1, 0, 3]]
    x = torch.tensor([[-800.0, -790.0, 0.0, -1000.0, -900.0, -900.0]], device=DEV)
    assert host(check(x, 4, groups=3, keep=2, group_top=2).ids).tolist() == [[2, 1, 0, 3]]


@pytest.mark.parametrize("T, E", [(60, 1024), (60, 256), (200, 40)])
def test_softmax_keys_within_the_error_of_their_sum(T, E):
    """The bias evens out the scores to 2^-24 of one another, the largest score about a half."""
    g = np.random.default_rng(E)
    one = g.normal(size=E) * 2
    one[E // 3] = np.log(np.exp(np.delete(one, E // 3)).sum())
    x = torch.from_numpy(np.tile(one, (T, 1)) + g.normal(size=(T, 1))).to(DEV, torch.float32)
    s = ref.scores(host(x.double()), 0)
    bias = torch.from_numpy((0.6 - s[0]).astype(np.float32)).to(DEV)
    check(x, 6, bias=bias)
    check(x, 6, bias=bias - 0.6)


@pytest.mark.parametrize("top", [1, 2])
def test_all_groups_kept_are_no_groups(top):
    x = logits(50, 24, torch.float32, 15)
    x[::3, 5], x[1::3, 20] = float("nan"), float("inf")
    r, one = s3r.route(x, 4, groups=4, keep=4, group_top=top), s3r.route(x, 4)
    assert torch.equal(r.ids, one.ids) and torch.equal(r.row_slot, one.row_slot)
    np.testing.assert_array_equal(host(r.ids), ref.choose(host(x), 4, groups=4, keep=4, group_top=top))


# ------------------------------------------------------------------ rows ----

def slots(T, k, R, seed):
    """A permutation's start: every slot a row of its own, some rows without a slot when R > T k."""
    p = np.random.default_rng(seed).permutation(max(R, T * k))[:T * k].reshape(T, k)
    return torch.from_numpy(p.astype(np.int32)).to(DEV)


ROWS = [(1, 1, 1, torch.bfloat16), (5, 2, 64, torch.bfloat16), (33, 8, 100, torch.float32), (64, 3, 2048, torch.bfloat16),
        (20, 2, 1411, torch.bfloat16), (17, 20, 520, torch.float32), (9, 1, 3, torch.float32)]


def half(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T, k, D, dtype", ROWS)
def test_combine(T, k, D, dtype, weighted):
    g = torch.Generator(DEV).manual_seed(T)
    sr = slots(T, k, T * k, T)
    rows = torch.randn(T * k, D, device=DEV, generator=g).to(dtype)
    w = torch.rand(T, k, device=DEV, generator=g) if weighted else None
    y = torch.empty(T, D, dtype=dtype, device=DEV)
    s3r.s3r_combine(rows, sr, w, y)
    exp, mag = ref.combine(host(rows.double()), host(sr), None if w is None else host(w))
    assert (np.abs(host(y.double()) - exp) <= (k + 1) * U * mag + half(dtype) * np.abs(exp) * (1 + 1e-6)).all()


@pytest.mark.parametrize("T, k, D, dtype", ROWS)
def test_dispatch_and_combine_backward(T, k, D, dtype):
    g = torch.Generator(DEV).manual_seed(T)
    R = T * k + 3
    sr = slots(T, k, R, T)
    x = torch.randn(T, D, device=DEV, generator=g).to(dtype)
    rows = torch.full((R, D), 9.0, dtype=dtype, device=DEV)
    s3r.s3r_dispatch(x, sr, rows)
    left = np.setdiff1d(np.arange(R), host(sr))
    for j in range(k):
        assert torch.equal(rows[sr[:, j].long()], x)
    assert (rows[left] == 9).all()
    rows = torch.randn(R, D, device=DEV, generator=g).to(dtype)
    w = torch.rand(T, k, device=DEV, generator=g)
    drows, dw = torch.full((R, D), 9.0, dtype=dtype, device=DEV), torch.empty(T, k, device=DEV)
    s3r.s3r_combine_backward(x, rows, sr, w, drows, dw)
    exp, edw, mag = ref.combine_backward(host(x.double()), host(rows.double()), host(sr), host(w))
    got = host(drows.double())
    on = np.isfinite(exp).all(axis=1)
    assert (got[~on] == 9).all()
    assert (np.abs(got - exp)[on] <= (U + half(dtype) * (1 + 1e-6)) * np.abs(exp)[on]).all()
    assert (np.abs(host(dw) - edw) <= (D + 8) * U * mag).all()


def test_slots_without_a_row():
    sr = torch.tensor([[0, -1], [7, 1], [-5, 1 << 30]], dtype=torch.int32, device=DEV)
    x = torch.randn(3, 16, device=DEV)
    rows = torch.zeros(4, 16, device=DEV)
    s3r.s3r_dispatch(x, sr, rows)
    assert torch.equal(rows, torch.stack([x[0], x[1], torch.zeros_like(x[0]), torch.zeros_like(x[0])]))
    y = torch.empty(3, 16, device=DEV)
    w = torch.full((3, 2), 2.0, device=DEV)
    s3r.s3r_combine(rows, sr, w, y)
    assert torch.equal(y, torch.stack([2 * x[0], 2 * x[1], torch.zeros_like(x[0])]))
    d, dw = torch.zeros(4, 16, device=DEV), torch.full((3, 2), 5.0, device=DEV)
    s3r.s3r_combine_backward(x, rows, sr, w, d, dw)
    assert torch.equal(d[:2], 2 * x[:2]) and (d[2:] == 0).all()
    assert host(dw)[[0, 1, 2, 2], [1, 0, 0, 1]].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("extra", [0, 5])
def test_gradient_of_rows_past_the_slots(extra):
    """More rows than slots: the helper's gradient of the others is 0, whatever its memory held."""
    T, k, D = 12, 2, 40
    r = s3r.route(logits(T, 8, torch.float32, 1), k)
    rows = torch.randn(T * k + extra, D, device=DEV)
    dy = torch.randn(T, D, device=DEV)
    for _ in range(3):
        torch.full_like(rows, float("nan"))              # left in the memory that is taken next
        drows, dw = s3r.combine_backward(dy, rows, r)
        exp, edw, mag = ref.combine_backward(host(dy), host(rows), host(r.slot_row), host(r.weights))
        assert (host(drows)[T * k:] == 0).all() and np.isfinite(exp[:T * k]).all()
        assert (np.abs(host(drows) - exp)[:T * k] <= U * np.abs(exp[:T * k])).all()
        assert (np.abs(host(dw) - edw) <= (D + 8) * U * mag).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_rows_of_every_width(dtype, offset):
    """Row ends at every place of a 16-byte word; nothing around the rows is read into them or written."""
    T, k = 7, 3
    sr = slots(T, k, T * k, 1)
    w = torch.rand(T, k, device=DEV)

    def inside(n, D, fill=None):
        wide = torch.full((n + 2, D + 21), 9.0 if fill is None else float("nan"), dtype=dtype, device=DEV)
        rows = wide[1:n + 1, offset:offset + D]
        if fill is not None:
            rows.copy_(fill)
        return wide, rows

    for D in [*range(1, 26), 511, 513, 515, 1029]:
        _, x = inside(T, D, torch.randn(T, D, device=DEV))
        _, rows = inside(T * k, D, torch.randn(T * k, D, device=DEV))
        wide, out = inside(T * k, D)
        s3r.s3r_dispatch(x, sr, out)
        assert all(torch.equal(out[sr[:, j].long()], x) for j in range(k))
        assert (wide == 9).sum() >= wide.numel() - out.numel()
        wide, y = inside(T, D)
        s3r.s3r_combine(rows, sr, w, y)
        exp, mag = ref.combine(host(rows.double()), host(sr), host(w))
        assert (np.abs(host(y.double()) - exp) <= (k + 1) * U * mag + half(dtype) * np.abs(exp) * (1 + 1e-6)).all()
        assert (wide == 9).sum() >= wide.numel() - y.numel()
        wide, d = inside(T * k, D)
        dw = torch.empty_like(w)
        s3r.s3r_combine_backward(x, rows, sr, w, d, dw)
        exp, edw, mag = ref.combine_backward(host(x.double()), host(rows.double()), host(sr), host(w))
        assert (np.abs(host(d.double()) - exp) <= (U + half(dtype) * (1 + 1e-6)) * np.abs(exp)).all()
        assert (np.abs(host(dw) - edw) <= (D + 8) * U * mag).all()
        assert (wide == 9).sum() >= wide.numel() - d.numel()


@pytest.mark.parametrize("T, D", [(2 ** 21 + 5, 2049), (2 ** 26 + 7, 8)])
def test_rows_past_32_bits(T, D):
    """More than 2^32 elements in odd rows; more tokens than a grid's dimension has waves."""
    x = ((torch.arange(T, device=DEV, dtype=torch.int32) % 127)[:, None].to(torch.bfloat16)
         + (torch.arange(D, device=DEV, dtype=torch.int32) % 63).to(torch.bfloat16))          # exact, below 2^8
    sr = torch.arange(T - 1, -1, -1, device=DEV, dtype=torch.int32)[:, None].contiguous()
    rows = torch.empty_like(x)
    s3r.s3r_dispatch(x, sr, rows)
    last = [0, 1, T // 2, T - 2, T - 1]
    part = torch.arange(0, T, 4099, device=DEV)
    for at in (part, torch.tensor(last, device=DEV)):
        assert torch.equal(rows[T - 1 - at], x[at])
    w = torch.full((T, 1), 2.0, device=DEV)
    y = torch.empty_like(x)
    s3r.s3r_combine(rows, sr, w, y)
    for at in (part, torch.tensor(last, device=DEV)):
        assert torch.equal(y[at], 2 * x[at])
    drows, dw = y, torch.empty_like(w)
    s3r.s3r_combine_backward(x, rows, sr, w, drows, dw)
    for at in (part, torch.tensor(last, device=DEV)):
        assert torch.equal(drows[T - 1 - at], 2 * x[at])
        exp = (x[at].double() ** 2).sum(1)                 # terms of one sign, D roundings of at most U each
        assert ((dw[at, 0].double() - exp).abs() <= (D + 8) * U * exp).all()


def test_route_backward_past_32_bits():
    T, E = 2 ** 29 + 9, 8                                   # 8 lanes a token: more than 2^32 of them
    x = (torch.arange(T, device=DEV, dtype=torch.int32) % 61)[:, None].to(torch.bfloat16) / 16 * torch.arange(
        E, device=DEV).to(torch.bfloat16)
    ids = torch.full((T, 1), 3, dtype=torch.int32, device=DEV)
    dw = torch.ones(T, 1, device=DEV)
    dx = torch.empty_like(x)
    s3r.s3r_route_backward(s3r.route_desc(T, E, 1, renorm=False), x, ids, dw, dx)
    at = torch.cat([torch.arange(0, T, 1048573, device=DEV), torch.arange(T - 70, T, device=DEV)])
    xs, chosen = host(x[at].double()), np.full((len(at), 1), 3)
    exp = ref.backward(xs, chosen, np.ones((len(at), 1)), renorm=False)
    # the softmax's exponentials and sums, |x| U and 16 roundings, on the scale of the gradient 1; half a bf16 step
    assert (np.abs(host(dx[at].double()) - exp) <= U * (64 + 2 * np.abs(xs).max()) + half(torch.bfloat16) * np.abs(exp)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_strides(dtype):
    T, k, D = 10, 2, 48
    sr = slots(T, k, T * k, 5)
    big = torch.randn(T * k, 100, device=DEV).to(dtype)
    xs = torch.randn(T, 100, device=DEV).to(dtype)
    w = torch.rand(T, k, device=DEV)
    for o in (0, 1, 8):
        rows, x = big[:, o:o + D], xs[:, o:o + D]
        y, yc = torch.zeros(T, 90, dtype=dtype, device=DEV), torch.empty(T, D, dtype=dtype, device=DEV)
        s3r.s3r_combine(rows, sr, w, y[:, 7:7 + D])
        s3r.s3r_combine(rows.contiguous(), sr, w, yc)
        assert torch.equal(y[:, 7:7 + D], yc) and (y[:, :7] == 0).all() and (y[:, 7 + D:] == 0).all()
        d, dw = torch.zeros_like(big), torch.empty_like(w)
        dc, dwc = torch.empty(T * k, D, dtype=dtype, device=DEV), torch.empty_like(w)
        s3r.s3r_combine_backward(x, rows, sr, w, d[:, o:o + D], dw)
        s3r.s3r_combine_backward(x.contiguous(), rows.contiguous(), sr, w, dc, dwc)
        assert torch.equal(d[:, o:o + D], dc)
        np.testing.assert_allclose(host(dw), host(dwc), atol=1e-3)      # another order of D bf16-sized products


def test_other_stream_and_graph_replays():
    """The calls record into a graph, and every replay gives the eager answer on changed inputs."""
    T, E, k, D = 700, 64, 2, 256
    x, rows = logits(T, E, torch.bfloat16, 12), torch.randn(T * k, D, device=DEV)
    d = s3r.route_desc(T, E, k)
    b = s3r.routed_buffers(d, DEV)
    y, dx = torch.empty(T, D, device=DEV), torch.empty_like(x)

    def step(stream=None):
        s3r.s3r_route(d, x, None, b.ids, b.weights, b.offsets, b.slot_row, b.row_slot, b.ws)
        s3r.s3r_combine(rows, b.slot_row, b.weights, y)
        s3r.s3r_route_backward(d, x, b.ids, b.weights, dx)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(logits(T, E, torch.bfloat16, 20 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (b.ids, b.weights, b.offsets, b.slot_row, b.row_slot, y, dx)]
        step()
        torch.cuda.synchronize()
        for g, e in zip(got, (b.ids, b.weights, b.offsets, b.slot_row, b.row_slot, y, dx)):
            assert torch.equal(g, e)
