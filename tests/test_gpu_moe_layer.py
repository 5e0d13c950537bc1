"""The mixture-of-experts layer (moe.py): its calls together, on an MI355X.

The forward pass against float64 on the values that the 4-bit codes stand for; the gradients, which pass
two quantizations, by their direction against the unquantized layer's.
"""
import numpy as np
import pytest
import torch

from oracle import mx, route
from stochastic_rounding_quantization_amd import moe, s3r
from tests._gpu import DEV, host

pytestmark = pytest.mark.gpu
T, E, K, D, F = 150, 6, 2, 256, 192


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)


@pytest.fixture(scope="module")
def step():
    g = torch.Generator(DEV).manual_seed(1)
    layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K)
    x, logits, dy = normal(g, T, D), normal(g, T, E), normal(g, T, D, std=1e-2)
    y, saved = layer.forward(x, logits)
    grads = layer.backward(saved, dy)
    torch.cuda.synchronize()
    return layer, x, logits, dy, y, saved, grads


def f(t):
    return host(t.float())


def test_forward(step):
    layer, x, logits, _, y, saved, _ = step
    ids = route.choose(f(logits), K)
    np.testing.assert_array_equal(host(saved.routed.ids), ids)
    offsets, slot_row, row_slot = route.order(ids, E)
    xq = mx.rows(f(x))["deq"][row_slot // K]
    a, rows = f(saved.gate_up), f(saved.rows)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        w = mx.rows(f(layer.gate_up[e]))["deq"]
        exp = xq[r] @ w.T
        assert (np.abs(a[r] - exp) <= 2.0 ** -8 * np.abs(exp) + D * 2.0 ** -23 * (np.abs(xq[r]) @ np.abs(w).T)).all()
        # the down product from the pre-activations that the layer kept: silu in fp64 may round to the other
        # neighbour of a code's border, one spacing of the block, so this is a bound on all of them together
        g, u = a[r, :F].astype(np.float64), a[r, F:].astype(np.float64)
        h = mx.rows((g / (1 + np.exp(-g)) * u).astype(np.float32))["deq"]
        exp = h @ mx.rows(f(layer.down[e]))["deq"].T
        assert np.linalg.norm(rows[r] - exp) <= 2.0 ** -7 * np.linalg.norm(exp)
    w = route.weights(f(logits), ids)
    exp, _ = route.combine(rows, slot_row, w)
    assert (np.abs(f(y) - exp) <= 2.0 ** -8 * np.abs(exp) + 2.0 ** -18 * np.abs(exp).max()).all()


def test_gradients_point_the_unquantized_way(step):
    layer, x, logits, dy, _, saved, grads = step
    xs, ls, wg, wd = (t.float().detach().requires_grad_() for t in (x, logits, layer.gate_up, layer.down))
    ids = saved.routed.ids.long()
    p = torch.softmax(ls, 1).gather(1, ids)
    p = p / p.sum(1, keepdim=True)
    y = torch.zeros(T, D, device=DEV)
    for e in range(E):
        t, j = torch.where(ids == e)
        a = xs[t] @ wg[e].t()
        h = torch.nn.functional.silu(a[:, :F]) * a[:, F:]
        y = y.index_add(0, t, p[t, j, None] * (h @ wd[e].t()))
    y.backward(dy.float())
    for got, exp in zip(grads, (xs.grad, ls.grad, wg.grad, wd.grad)):
        got = got.float()
        assert got.shape == exp.shape and torch.isfinite(got).all()
        cos = torch.nn.functional.cosine_similarity(got.flatten(), exp.flatten(), dim=0)
        assert cos > 0.95, float(cos)


def test_empty_batch_and_one_token(step):
    layer, x, logits = step[:3]
    y, _ = layer.forward(x[:1], logits[:1])
    full = step[4]
    # one token's rows go another way through the product kernels: the order of fp32 sums may differ, then bf16
    assert (np.abs(f(y) - f(full[:1])) <= 2.0 ** -6 * np.abs(f(full[:1])).max()).all()
    assert layer.forward(x[:0], logits[:0])[0].shape == (0, D)


# ---------------------------------------------------- gradients, by size ----

def gradients(layer, x, logits, saved, dy, scale):
    """The layer's gradients in float64 at the values that its forward pass kept: dx, dlogits, dgate_up, ddown."""
    x, logits, dy, a, rows = (t.double().cpu() for t in (x, logits, dy, saved.gate_up, saved.rows))
    wg, wd = layer.gate_up.double().cpu(), layer.down.double().cpu()
    r = saved.routed
    o, slot = r.offsets.tolist(), r.row_slot.long().cpu()
    tok = slot // layer.top_k
    w = torch.from_numpy(route.weights(logits.numpy(), host(r.ids), scale=scale)).reshape(-1)
    drows = w[slot, None] * dy[tok]
    dw = (dy[tok] * rows).sum(1)
    dweights = torch.empty_like(w)
    dweights[slot] = dw
    dlogits = route.backward(logits.numpy(), host(r.ids), dweights.reshape(r.ids.shape).numpy(), scale=scale)
    dx, dgu, dd = torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wd)
    for e in range(wg.shape[0]):
        s = slice(o[e], o[e + 1])
        g, u = a[s, :layer.ff], a[s, layer.ff:]
        sg = torch.sigmoid(g)
        dh = drows[s] @ wd[e]
        dd[e] = drows[s].t() @ (g * sg * u)
        da = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1)
        dgu[e] = da.t() @ x[tok[s]]
        dx.index_add_(0, tok[s], da @ wg[e])
    return dx, torch.from_numpy(dlogits), dgu, dd


def close(got, exp, bound):
    """Relative error of the whole tensor and its length."""
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    assert (got - exp).norm() <= bound * exp.norm(), float((got - exp).norm() / exp.norm())
    assert abs(got.norm() / exp.norm() - 1) <= bound


# What is left is the INT8 rounding.  An expert's gradients are rounded to 127 steps of their largest magnitude, about
# 10 times their root mean square (products of two normal factors): stochastic rounding errs by 0.41 of a step, 10 / 127 *
# 0.41 = 3 %; the INT8 rows and weights (4 / 127 * 0.29 = 1 %) and bf16 (0.2 %) add little, and a second product doubles
# the square of it: under 5 % for dx, dgate and dup.  Twice that is the bound; a factor or a term that is missing is more.
BOUND = 0.1


@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_gradients_by_expert(scale):
    g = torch.Generator(DEV).manual_seed(5)
    n, none = 300, 3
    layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K, scale=scale)
    x, logits, dy = normal(g, n, D), normal(g, n, E), normal(g, n, D, std=1e-2)
    logits[:, none] = float("-inf")                      # an expert without a row
    y, saved = layer.forward(x, logits)
    dx, dlogits, dgu, dd = layer.backward(saved, dy)
    ex, el, egu, ed = gradients(layer, x, logits, saved, dy, scale)
    close(dx, ex, BOUND)
    # the router's gradient passes no rounding but fp32's and a bf16 result's: D additions of both weights' products, 2^-8
    mag = (dy.double().abs()[:, None].cpu() * saved.rows.double().abs().cpu()[saved.routed.slot_row.long().cpu()]).sum(2).amax(1)
    assert ((dlogits.double().cpu() - el).abs() <= 2 ** -8 * el.abs() + scale * (D + 80) * 2 ** -24 * mag[:, None]).all()
    for e in range(E):
        if e == none:
            assert (dgu[e] == 0).all() and (dd[e] == 0).all()
        else:
            close(dgu[e, :F], egu[e, :F], BOUND)
            close(dgu[e, F:], egu[e, F:], BOUND)
            close(dd[e], ed[e], BOUND)



def test_gradients_without_tokens(step):
    layer, x, logits, dy = step[:4]
    y, saved = layer.forward(x[:0], logits[:0])
    dx, dlogits, dgu, dd = layer.backward(saved, dy[:0])
    assert dx.shape == (0, D) and dlogits.shape == (0, E) and dx.dtype == dgu.dtype == dd.dtype == torch.float32
    assert dgu.shape == layer.gate_up.shape and dd.shape == layer.down.shape and (dgu == 0).all() and (dd == 0).all()
    assert dlogits.dtype == logits.dtype


# ------------------------------------------------------- changed weights ----

def fresh(layer):
    return moe.MoeLayer(layer.gate_up.clone(), layer.down.clone(), layer.top_k, **layer.router)


def same_step(layer, x, logits, dy, other=None):
    """A training step of the layer has the bits of one of a layer made anew from its weights."""
    other = other or fresh(layer)
    y, saved = layer.forward(x, logits)
    got = y, *layer.backward(saved, dy)
    y, saved = other.forward(x, logits)
    return all(torch.equal(a, b) for a, b in zip(got, (y, *other.backward(saved, dy))))


def test_weights_changed_in_place(step):
    """As an optimizer does between two steps, and once between construction and the first backward pass."""
    g = torch.Generator(DEV).manual_seed(6)
    x, logits, dy = step[1:4]
    layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K)
    layer.gate_up.mul_(1.5)
    assert same_step(layer, x, logits, dy)
    layer.down.add_(normal(g, E, D, F, std=0.1))
    assert same_step(layer, x, logits, dy)
    layer.gate_up.sub_(normal(g, E, 2 * F, D, std=0.1))
    layer.down.mul_(-1)
    assert same_step(layer, x, logits, dy)
    layer.down = normal(g, E, D, F, std=0.1)             # another tensor
    assert same_step(layer, x, logits, dy)


def test_weights_changed_unseen(step):
    """Through .data, which torch does not count: the codes follow the call that says so."""
    g = torch.Generator(DEV).manual_seed(7)
    x, logits, dy = step[1:4]
    layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K)
    assert same_step(layer, x, logits, dy)
    layer.gate_up.data.mul_(0.5)
    layer.down.data.mul_(-1)
    layer.weights_changed()
    assert same_step(layer, x, logits, dy)


def test_codes_for_another_stream(step):
    """A stream that did not make the codes waits for them: the second pass follows the first with no word between them."""
    g = torch.Generator(DEV).manual_seed(8)
    x, logits, dy = step[1:4]
    side = torch.cuda.Stream()
    for _ in range(3):
        layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K)
        other = fresh(layer)
        y, saved = other.forward(x, logits)
        want = y, *other.backward(saved, dy)
        for renewed in (False, True):
            if renewed:
                layer.gate_up.mul_(1.0)                  # the same values, made again
            torch.cuda.synchronize()
            torch.randn(1 << 24, device=DEV).sort()       # the codes of this stream's pass come after this
            y, saved = layer.forward(x, logits)
            layer.backward(saved, dy)
            with torch.cuda.stream(side):
                y, saved = layer.forward(x, logits)
                got = y, *layer.backward(saved, dy)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_codes_in_a_graph(step):
    """A graph takes the kept codes, which weights_changed renews in place, or makes its own of a weight changed since."""
    g = torch.Generator(DEV).manual_seed(9)
    x, logits = step[1:3]
    for changed in (False, True):
        layer = moe.MoeLayer(normal(g, E, 2 * F, D, std=0.1), normal(g, E, D, F, std=0.1), K)
        layer.forward(x, logits)
        if changed:
            layer.gate_up.mul_(1.5)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, _ = layer.forward(x, logits)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, fresh(layer).forward(x, logits)[0])
            assert torch.equal(y, layer.forward(x, logits)[0])
            layer.gate_up.mul_(1.5)
            layer.down.sub_(0.01)
            layer.weights_changed()
