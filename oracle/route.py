"""Routing to experts, its gradient, and the rows' way to the experts and back.  (Oracle: test use only.)

float64 throughout, row by row in plain Python where the order of decisions matters.
Definitions: include/s3r.h, "routing to experts" and "tokens to the experts' rows and back".
"""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(x, score):
    """s of every logit; a fully masked softmax row has zeros."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        z = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        total = z.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, z / total)


def _descending(key):
    """Indices by descending key, ties to the lower index; NaN ranks as -inf."""
    k = [(-v if v == v else np.inf) for v in key]
    return sorted(range(len(k)), key=lambda e: (k[e], e))


def choose(x, top_k, *, score=SOFTMAX, bias=None, groups=1, keep=1, group_top=1):
    """ids int32 [T x top_k]."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    if keep == groups:
        groups = 1
    masked = np.isneginf(x) | np.isnan(x)
    key = scores(x, score) + (0.0 if bias is None else np.asarray(bias, np.float64))
    key = np.where(masked | np.isnan(key), -np.inf, key)
    # without a bias the logits stand for the scores, wherever these are not added up: their order, also where fp64
    # scores meet
    by_logit = np.where(masked, -np.inf, x)
    group_key = by_logit if bias is None and group_top == 1 else key
    if bias is None:
        key = by_logit if groups == 1 or group_top == 1 else np.where(np.isneginf(key), -np.inf, x)
    per = E // groups
    ids = np.empty((T, top_k), np.int32)
    for t in range(T):
        k, g_key = key[t], group_key[t]
        if groups > 1:
            with np.errstate(invalid="ignore"):          # inf - inf: NaN
                of = [sum(sorted(g_key[g * per:(g + 1) * per], reverse=True)[:group_top]) for g in range(groups)]
            best = set(_descending(of)[:keep])
            k = np.array([k[e] if e // per in best else -np.inf for e in range(E)])
        ids[t] = _descending(k)[:top_k]
    return ids


def weights(x, ids, *, score=SOFTMAX, renorm=True, scale=1.0):
    x = np.asarray(x, np.float64)
    if not renorm:
        return scale * np.take_along_axis(scores(x, score), ids.astype(np.int64), axis=1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        xs = np.take_along_axis(x, ids.astype(np.int64), axis=1)
        log_s = -np.logaddexp(0.0, -xs) if score == SIGMOID else xs
        top = log_s.max(axis=1, keepdims=True)
        p = np.exp(log_s - np.where(np.isneginf(top), 0.0, top))
        total = p.sum(axis=1, keepdims=True)
        p = np.where(total == 0, 0.0, p / total)
        if score == SOFTMAX:
            odd = (np.isnan(x) | np.isposinf(x)).any(axis=1, keepdims=True)
            p = np.where(odd, np.nan, p)
        return scale * p


def order(ids, experts):
    """(offsets int64 [E + 1], slot_row int32 [T x k], row_slot int32 [T * k]): a bucket per expert, filled in slot order."""
    buckets = [[] for _ in range(experts)]
    for slot, e in enumerate(ids.reshape(-1)):
        buckets[e].append(slot)
    row_slot = np.array([s for b in buckets for s in b], np.int32)
    offsets = np.concatenate([[0], np.cumsum([len(b) for b in buckets])]).astype(np.int64)
    slot_row = np.empty(ids.size, np.int32)
    slot_row[row_slot] = np.arange(ids.size, dtype=np.int32)
    return offsets, slot_row.reshape(ids.shape), row_slot


def backward(x, ids, dweights, *, score=SOFTMAX, renorm=True, scale=1.0):
    """dlogits [T x E], by the chain rule through the scores; ids outside 0 .. E-1 take no part."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    out = np.zeros((T, E))
    with np.errstate(over="ignore", invalid="ignore"):   # a NaN or +inf among the chosen leaves NaN
        _backward_rows(out, x, ids, dweights, score, renorm, scale)
    return out


def _backward_rows(out, x, ids, dweights, score, renorm, scale):
    T, E = x.shape
    for t in range(T):
        at = [j for j, e in enumerate(ids[t]) if 0 <= e < E]
        e = ids[t][at].astype(np.int64)
        g = np.asarray(dweights[t], np.float64)[at] * scale
        if renorm:
            # p_j of the chosen, from their log scores; dp/dlog s = p (g - <p, g>)
            log_s = -np.logaddexp(0.0, -x[t, e]) if score == SIGMOID else x[t, e]
            top = log_s.max() if len(e) else -np.inf
            p = np.exp(log_s - top) if top != -np.inf else np.zeros(len(e))
            p = p / p.sum() if p.sum() != 0 else p
            d = p * (g - (p * g).sum())
            out[t, e] = d * np.exp(-np.logaddexp(0.0, x[t, e])) if score == SIGMOID else d
        else:
            s = scores(x[t:t + 1], score)[0]
            if score == SIGMOID:
                out[t, e] = g * s[e] * np.exp(-np.logaddexp(0.0, x[t, e]))
            else:
                spread = np.zeros(E)
                spread[e] = g
                out[t] = s * (spread - (g * s[e]).sum())


def combine(rows, slot_row, w=None):
    """(y, sum of |w| |row|) float64; slots without a row add nothing."""
    rows = np.asarray(rows, np.float64)
    T, k = slot_row.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < rows.shape[0]:
                f = 1.0 if w is None else float(w[t, j])
                y[t] += f * rows[r]
                mag[t] += abs(f) * np.abs(rows[r])
    return y, mag


def combine_backward(dy, rows, slot_row, w):
    """(drows with NaN where no slot leads, dw, sum of |dy| |row|)."""
    dy, rows = np.asarray(dy, np.float64), np.asarray(rows, np.float64)
    T, k = slot_row.shape
    drows = np.full(rows.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < rows.shape[0]:
                drows[r] = float(w[t, j]) * dy[t]
                dw[t, j] = (dy[t] * rows[r]).sum()
                mag[t, j] = (np.abs(dy[t]) * np.abs(rows[r])).sum()
    return drows, dw, mag
