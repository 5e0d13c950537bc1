"""Refusals of the orthogonalised update (host checks, before any HIP call), and pins of its oracle.

Pointers are invented, aligned addresses: a call that passed its checks would return the architecture's
error here (there is no GPU) or S3R_ERR_HIP, never S3R_OK; each test first shows that its base call gets that far.
"""
import ctypes

import numpy as np
import pytest

from oracle import orth
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


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw, rc", [
    (dict(shape=(-1, 4, 4)), INVALID), (dict(shape=(65536, 4, 4)), INVALID), (dict(shape=(1 << 20, 4)), INVALID),
    (dict(shape=(4, 1 << 20)), INVALID), (dict(shape=(-4, 4)), INVALID), (dict(steps=0), INVALID), (dict(steps=65), INVALID),
    (dict(coeffs=(NAN, 1, 1)), INVALID), (dict(coeffs=(1, INF, 1)), INVALID), (dict(coeffs=(1, 1, -INF)), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(scale=INF), INVALID), (dict(keep=NAN), INVALID),
    (dict(reserved=1), INVALID), (dict(g_dtype=2), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED), (dict(G=None), INVALID),
    (dict(G=P + 2), INVALID), (dict(out=None), INVALID), (dict(out=P + 1), INVALID), (dict(ld=49), INVALID), (dict(ld_out=49), INVALID),
    (dict(shape=(2, 30, 50), g_stride=1499), INVALID), (dict(shape=(2, 30, 50), out_stride=1499), INVALID),
    (dict(G=2 * P, out_dtype=1), INVALID), (dict(G=2 * P, ld=51), INVALID),
    (dict(G=2 * P, shape=(2, 30, 50), g_stride=1501), INVALID),
    (dict(ws=None), INVALID), (dict(ws=P + 128), INVALID), (dict(wsb=4096), WORKSPACE)])
def test_refuses(L, kw, rc):
    def call(shape=(30, 50), G=P, ld=50, g_stride=1500, out=2 * P, ld_out=50, out_stride=1500, ws=P, wsb=1 << 30, reserved=0, **d):
        desc = s3r.orth_desc(shape, d.pop("g_dtype", 0), d.pop("out_dtype", 0), **d)
        desc.reserved = reserved
        return L.s3r_orthogonalize(ctypes.byref(desc), G, ld, g_stride, out, ld_out, out_stride, ws, wsb, None)
    assert call() in PAST and call(shape=(2, 30, 50)) in PAST and call(G=2 * P) in PAST and call(out_dtype=1, g_dtype=1) in PAST
    assert call(shape=(0, 50), G=None, out=None) in PAST
    assert call(**kw) == rc


def test_workspace(L):
    assert s3r.s3r_orthogonalize_workspace(s3r.orth_desc((0, 7))) == 256
    assert s3r.s3r_orthogonalize_workspace(s3r.orth_desc((3, 7), steps=0)) == 0
    big = s3r.s3r_orthogonalize_workspace(s3r.orth_desc((64, 1408, 2048)))
    assert 64 * 1408 * 2048 * 12 < big < 64 * 1408 * 2048 * 24
    assert L.s3r_orthogonalize(None, P, 5, 5, P, 5, 5, P, 1 << 30, None) == INVALID


def test_binding_checks_tensors(L):
    import torch
    G = torch.zeros(4, 6)
    ws = s3r.orthogonalize_buffer(G)
    for call in (lambda: s3r.s3r_orthogonalize(G, torch.zeros(4, 5), ws=ws), lambda: s3r.s3r_orthogonalize(G.t(), torch.zeros(6, 4), ws=ws),
                 lambda: s3r.s3r_orthogonalize(G, G.half(), ws=ws), lambda: s3r.s3r_orthogonalize(G[0], G[0], ws=ws),
                 lambda: s3r.s3r_orthogonalize(G.long(), G, ws=ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(s3r.S3RError):
        s3r.s3r_orthogonalize(G, G.clone(), ws=None, stream=0)


def test_oracle_follows_the_singular_values():
    """The steps keep the singular vectors and take each singular value through a s + b s^3 + c s^5."""
    r = np.random.default_rng(1)
    for shape in ((9, 14), (14, 9)):
        G = r.normal(size=shape)
        U, s, V = np.linalg.svd(G, full_matrices=False)
        s = s / (np.sqrt((s * s).sum()) + np.float64(np.float32(1e-7)))
        a, b, c = (np.float64(np.float32(v)) for v in orth.COEFFS)
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        np.testing.assert_allclose(orth.newton_schulz(G), (U * s) @ V, atol=1e-12)
    assert not orth.newton_schulz(np.zeros((3, 4)), eps=0.0).any()


@pytest.fixture
def launches(L, monkeypatch):
    """The binding up to the launch, which does nothing here: (u, W, arguments) of each."""
    import torch
    seen, real = [], s3r.s3r_orthogonalize

    def call(u, W, **kw):
        seen.append((u.clone(), W, kw))
        assert real(u, W, **kw, stream=0, rc_only=True) in PAST
        W.add_(1)                                  # as if written
    monkeypatch.setattr(s3r, "s3r_orthogonalize", call)

    def aligned(nbytes, device):
        ws = torch.empty(nbytes + 256, dtype=torch.uint8)
        return ws[-ws.data_ptr() % 256:][:nbytes]
    monkeypatch.setattr(s3r, "_scratch", aligned)
    return seen


def muon(nesterov=True, **kw):
    import torch
    from stochastic_rounding_quantization_amd.optim import Muon
    g = torch.Generator().manual_seed(1)
    weights = [torch.randn(4, 6, generator=g), torch.randn(2, 5, 3, generator=g).bfloat16()]
    grads = [torch.randn(W.shape, generator=g) for W in weights]
    return Muon(weights, lr=0.1, nesterov=nesterov, **kw), weights, grads


def column_major(t):
    return t.transpose(-1, -2).contiguous().transpose(-1, -2)


@pytest.mark.parametrize("nesterov", [True, False])
def test_optimizer_takes_gradients_of_any_layout(launches, nesterov):
    """A column-major gradient, a bf16 one and a slice give the update of the same numbers in a row."""
    import torch
    for other in (column_major, lambda g: torch.cat([g, g], -1)[..., :g.shape[-1]], lambda g: g):
        for dtype in (torch.float32, torch.bfloat16):
            del launches[:]
            for layout in (lambda g: g, other):
                opt, _, grads = muon(nesterov)
                for _ in range(2):
                    opt.step([layout(g.to(dtype)) for g in grads])
                launches.append(opt.buffers)
            half = len(launches) // 2
            assert half == 5
            for a, b in zip(launches[:4], launches[half:-1]):
                assert torch.equal(a[0], b[0]) and a[0].is_contiguous()
            assert all(torch.equal(a, b) for a, b in zip(launches[4], launches[-1]))
    opt, _, grads = muon(nesterov)
    del launches[:]
    opt.step(grads)
    opt.step([2 * g for g in grads])
    buf = 0.95 * grads[0] + 2 * grads[0]
    torch.testing.assert_close(launches[2][0], 2 * grads[0] + 0.95 * buf if nesterov else buf)


@pytest.mark.parametrize("what", ["gradient shape", "one gradient", "gradient device", "rate", "decay", "steps",
                                  "coefficients", "weight layout", "weight type", "weight device"])
def test_refused_steps_change_nothing(launches, what):
    import torch
    opt, weights, grads = muon()
    opt.step(grads)
    del launches[:]
    before = [t.clone() for t in (*weights, *opt.buffers)]
    if what == "gradient shape":
        grads[1] = grads[1].transpose(1, 2)
    elif what == "one gradient":
        grads.pop()
    elif what == "gradient device":
        grads[1] = grads[1].to("meta")
    elif what == "rate":
        opt.lr = NAN
    elif what == "decay":
        opt.decay = 1e300
    elif what == "steps":
        opt.steps = 65
    elif what == "coefficients":
        opt.coeffs = (1.0, INF, 0.0)
    elif what == "weight layout":
        opt.weights[1] = column_major(weights[1])
    elif what == "weight type":
        opt.weights[1] = weights[1].half()
    else:
        opt.weights[1] = weights[1].to("meta")
    with pytest.raises(ValueError):
        opt.step(grads)
    assert not launches
    assert all(torch.equal(a, b) for a, b in zip(before, (*weights, *opt.buffers)))


def test_optimizer_refuses_weights_that_no_step_takes():
    import torch
    from stochastic_rounding_quantization_amd.optim import Muon
    W = torch.zeros(4, 6)
    for bad in (W.t(), W[0], W.half(), W.double(), torch.zeros(2, 2, 4, 6), W[:, ::2], W[:1].expand(4, 6), torch.zeros(1, 4, 6).expand(2, 4, 6)):
        with pytest.raises(ValueError):
            Muon([W.clone(), bad], lr=0.1)
    Muon([], lr=0.1).step([])
    for good in (W, W[:, 1:4], torch.zeros(2, 4, 6)[:, 1:3], torch.zeros(0, 6), torch.zeros(3, 0, 2)):
        Muon([good], lr=0.1)


@pytest.mark.parametrize("coeffs", [(1.0, -0.5), (1.0, 2.0, 3.0, 4.0), ()])
def test_binding_takes_three_coefficients(L, coeffs):
    """Two would have left the others a place off: eps as c, scale as eps, a result of zeros."""
    import torch
    from stochastic_rounding_quantization_amd.optim import Muon
    G = torch.zeros(4, 6)
    for call in (lambda: s3r.orth_desc((4, 6), coeffs=coeffs), lambda: s3r.s3r_orthogonalize(G, G.clone(), coeffs=coeffs, stream=0),
                 lambda: Muon([G], lr=0.1, coeffs=coeffs)):
        with pytest.raises(ValueError):
            call()
