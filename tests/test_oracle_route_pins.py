"""Pins of the routing oracle (oracle/route.py): closed forms, torch's own functions, differences."""
import numpy as np
import pytest
import torch

from oracle import mx, route


@pytest.mark.parametrize("score", [route.SOFTMAX, route.SIGMOID])
def test_scores_against_torch(score):
    x = np.random.default_rng(1).normal(size=(7, 13)) * 4
    t = torch.from_numpy(x)
    exp = torch.softmax(t, 1) if score == route.SOFTMAX else torch.sigmoid(t)
    np.testing.assert_allclose(route.scores(x, score), exp.numpy(), rtol=1e-13)


def test_choice_is_topk_without_ties_and_lowest_index_with():
    x = np.random.default_rng(2).normal(size=(50, 20))
    np.testing.assert_array_equal(route.choose(x, 4), torch.topk(torch.from_numpy(x), 4).indices.numpy())
    assert route.choose(np.zeros((1, 6)), 3).tolist() == [[0, 1, 2]]
    assert route.choose(np.array([[1.0, 3.0, 3.0, 2.0]]), 3).tolist() == [[1, 2, 3]]


def test_masked_experts_come_last():
    x = np.array([[-np.inf, 1.0, -np.inf, 2.0], [-np.inf] * 4, [np.nan, 0.0, -1.0, -2.0]])
    assert route.choose(x, 3).tolist() == [[3, 1, 0], [0, 1, 2], [1, 2, 3]]
    w = route.weights(x[:2], np.array([[3, 1, 0], [0, 1, 2]]))
    np.testing.assert_allclose(w[0], [np.e / (1 + np.e), 1 / (1 + np.e), 0.0])
    assert w[1].tolist() == [0, 0, 0]


def test_groups_by_hand():
    # groups {0,1} {2,3} {4,5}: largest 5, 4, 4.5; sums of two 5.1, 7.9, 8.0
    x = np.array([[5.0, 0.1, 4.0, 3.9, 4.5, 3.5]])
    assert route.choose(x, 2, groups=3, keep=1).tolist() == [[0, 1]]
    s = np.log(x / 6) - np.log(1 - x / 6)             # sigmoid keys x / 6
    assert route.choose(s, 2, score=route.SIGMOID, groups=3, keep=1, group_top=2).tolist() == [[4, 5]]
    assert route.choose(s, 2, score=route.SIGMOID, groups=3, keep=2, group_top=2).tolist() == [[4, 2]]
    assert route.choose(s, 2, score=route.SIGMOID, groups=3, keep=1, group_top=2,
                        bias=[0, 0, 0, 0.1, 0, 0]).tolist() == [[3, 2]]


def test_order_is_a_stable_sort():
    ids = np.random.default_rng(3).integers(0, 5, (40, 3)).astype(np.int32)
    offsets, slot_row, row_slot = route.order(ids, 6)
    np.testing.assert_array_equal(row_slot, np.argsort(ids.reshape(-1), kind="stable"))
    np.testing.assert_array_equal(slot_row.reshape(-1)[row_slot], np.arange(120))
    assert offsets.tolist()[-2:] == [120, 120] and offsets[0] == 0


@pytest.mark.parametrize("score", [route.SOFTMAX, route.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(4)
    x, g = rng.normal(size=(3, 8)), rng.normal(size=(3, 3))
    ids = route.choose(x, 3)
    d = route.backward(x, ids, g, score=score, renorm=renorm, scale=1.5)
    h = 1e-5
    for t in range(3):
        for e in range(8):
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            f = [(route.weights(v, ids, score=score, renorm=renorm, scale=1.5) * g).sum() for v in (up, dn)]
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) < 1e-8       # h^2 and 2^-53 / h


def test_combine_is_the_transpose_of_its_gradient():
    rng = np.random.default_rng(5)
    slot_row = rng.permutation(12).reshape(6, 2).astype(np.int32)
    slot_row[2, 1] = -1
    rows, dy, w = rng.normal(size=(12, 5)), rng.normal(size=(6, 5)), rng.normal(size=(6, 2))
    y, _ = route.combine(rows, slot_row, w)
    drows, dw, _ = route.combine_backward(dy, rows, slot_row, w)
    np.testing.assert_allclose((y * dy).sum(), np.nansum(drows * rows))
    np.testing.assert_allclose((y * dy).sum(), (dw * w).sum())
    assert dw[2, 1] == 0


def test_mx_rows_pads_with_zeros():
    M = np.random.default_rng(6).normal(size=(3, 77)).astype(np.float32)
    q = mx.rows(M)
    assert q["codes"].shape == (3, 128) and (q["codes"][:, 77:] == 0).all() and (q["scale"][:, 3:] == 0).all()
    step = np.repeat(np.ldexp(1.0, q["scale"].astype(int) - 127), 32, axis=1)[:, :77]
    assert (np.abs(q["deq"] - M) <= step).all()           # half the widest spacing, 2


def test_two_largest_groups_choose_by_logits_where_scores_meet():
    """Without a bias the scores order the groups and the logits the experts in them: equal scores are no tie."""
    x = np.array([[40.0, 50.0, 0.0, 0.0]])                # both sigmoids are 1 in fp64
    assert route.choose(x, 1, score=route.SIGMOID, groups=2, keep=1, group_top=2).tolist() == [[1]]
    x = np.array([[-800.0, -790.0, 0.0, -1000.0, -900.0, -900.0]])    # all softmax scores but one are 0
    assert route.choose(x, 4, groups=3, keep=2, group_top=2).tolist() == [[2, 1, 0, 3]]
    x = np.array([[-800.0, np.nan, 0.0, -np.inf, 1.0, 2.0]])      # a NaN logit makes the row's scores NaN: all rank as -inf
    assert route.choose(x, 3, groups=3, keep=2, group_top=2).tolist() == [[0, 1, 2]]


def test_group_sum_of_both_infinities_ranks_last():
    b = np.array([np.inf, -np.inf, 0, 0, 1, 1])
    x = np.zeros((1, 6))
    assert route.choose(x, 2, bias=b, groups=3, keep=1, group_top=2).tolist() == [[4, 5]]
    assert route.choose(x, 4, bias=b, groups=3, keep=2, group_top=2).tolist() == [[4, 5, 2, 3]]


@pytest.mark.parametrize("score, odd", [(route.SOFTMAX, np.nan), (route.SOFTMAX, np.inf), (route.SIGMOID, np.nan)])
def test_gradient_of_a_chosen_nan(score, odd):
    x = np.array([[1.0, odd, 0.5, 2.0], [1.0, 3.0, 0.5, 2.0]])
    d = route.backward(x, np.array([[1, 3], [1, 3]], np.int32), np.ones((2, 2)), score=score)
    assert np.isnan(d[0, [1, 3]]).all() and (d[0, [0, 2]] == 0).all() and np.isfinite(d[1]).all()


def test_gradient_of_a_saturated_sigmoid_is_finite():
    d = route.backward(np.array([[np.inf, 0.0, -np.inf]]), np.array([[0, 1, 2]], np.int32), np.array([[1.0, 2.0, 3.0]]),
                       score=route.SIGMOID)
    np.testing.assert_allclose(d, [[0.0, (1 / 3) * (2 - 4 / 3) / 2, 0.0]])


@pytest.mark.parametrize("group_top", [1, 2])
def test_all_groups_kept_are_no_groups(group_top):
    """Also where the scores are NaN: without a bias the logits decide."""
    x = np.array([[1.0, np.nan, 0.5, 2.0], [1.0, np.inf, 0.5, 2.0], [0.0, 3.0, 0.5, 2.0]])
    assert route.choose(x, 3, groups=2, keep=2, group_top=group_top).tolist() == [[3, 0, 2], [1, 3, 0], [1, 3, 2]]
