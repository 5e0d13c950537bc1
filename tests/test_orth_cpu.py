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
