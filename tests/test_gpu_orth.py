"""Orthogonalised updates on an MI355X against oracle/orth.py in float64.

How far a result may be off, before any was seen: a value is kept to 2^-24 of itself in two planes of 11 bits, a product
leaves out 2^-24 of its terms and adds in fp32, a few 2^-24 of the running magnitudes more.  So the oracle runs again with
every stored value off by a normal error of 2^-22 of the magnitudes that went into it, and a result may be 4 times as far
(in the Frobenius norm) from the exact one, plus half a step of its type and what the planes' smallest step, 2^-37 of X's
largest possible singular value, comes to in the steps (which matters where eps leaves X tiny).
"""
import numpy as np
import pytest
import torch

from oracle import orth
from stochastic_rounding_quantization_amd import s3r
from tests._gpu import DEV, host

pytestmark = pytest.mark.gpu
BOTH = [torch.float32, torch.bfloat16]
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gradient(shape, dtype, seed, size=1e-4):
    """A few strong directions and noise."""
    r = np.random.default_rng(seed)
    *batch, N, K = shape
    k = min(4, N, K)
    x = r.normal(size=(*batch, N, k)) @ r.normal(size=(*batch, k, K)) + r.normal(size=shape)
    return torch.from_numpy(x * size).to(DEV, dtype)


def check(got, G, out=torch.float32, **kw):
    g = host(G.double())
    exp = orth.newton_schulz(g, **kw)
    far = orth.newton_schulz(g, noise=2.0 ** -22, **kw)
    floor = 2.0 ** -37 * max(1.0, abs(kw.get("coeffs", orth.COEFFS)[0])) ** kw.get("steps", 5) * np.sqrt(exp.size)
    most = 4 * np.linalg.norm(far - exp) + HALF[out] * np.linalg.norm(exp) + floor
    off = np.linalg.norm(host(got.double()) - exp)
    print(f"{tuple(G.shape)}: {off / max(np.linalg.norm(exp), 1e-300):.2e} of {most / max(np.linalg.norm(exp), 1e-300):.2e}")
    assert off <= most


SHAPES = [(1, 1), (1, 7), (7, 1), (16, 16), (31, 33), (33, 65), (64, 64), (65, 64), (100, 300), (300, 100), (3, 1000),
          (256, 512), (701, 1283), (1283, 701), (40, 5000), (200, 8192)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype):
    G = gradient(shape, dtype, shape[0])
    check(s3r.orthogonalize(G, out_dtype=torch.float32), G)
    check(s3r.orthogonalize(G, out_dtype=torch.bfloat16), G, torch.bfloat16)


@pytest.mark.parametrize("steps, coeffs, eps", [(1, orth.COEFFS, 1e-7), (2, (1.5, -0.5, 0.0), 1e-3), (9, (1.875, -1.25, 0.375), 0.0),
                                                (6, orth.COEFFS, 1.0), (3, (0.0, 1.0, 0.0), 1e-7)])
def test_steps_and_coefficients(steps, coeffs, eps):
    for shape in ((50, 120), (130, 70)):
        G = gradient(shape, torch.float32, steps)
        check(s3r.orthogonalize(G, steps=steps, coeffs=coeffs, eps=eps), G, steps=steps, coeffs=coeffs, eps=eps)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e36])
def test_sizes_of_values(size):
    """No square leaves its range, and what eps leaves of a tiny matrix is right."""
    G = gradient((70, 90), torch.float32, 3, size)
    check(s3r.orthogonalize(G, eps=0.0), G, eps=0.0)
    check(s3r.orthogonalize(G), G)


def test_several_matrices_strides_scale_and_keep():
    G = gradient((5, 70, 133), torch.float32, 1)
    for dtype in BOTH:
        each = torch.stack([s3r.orthogonalize(g, out_dtype=dtype) for g in G])
        wide = torch.full((5, 80, 140), 7.0, device=DEV).to(dtype)
        src = torch.full((5, 72, 150), float("nan"), device=DEV)
        src[:, 1:71, 3:136] = G
        out = wide[:, 5:75, 1:134]
        ws = s3r.orthogonalize_buffer(G)
        s3r.s3r_orthogonalize(src[:, 1:71, 3:136], out, ws=ws)
        assert torch.equal(out, each)
        s3r.s3r_orthogonalize(src[:, 1:71, 3:136], out, scale=-0.5, keep=0.25, ws=ws)
        exp, size = 0.25 * each.double() - 0.5 * each.double(), each.double().abs()
        # X lies within half a step of `each`, which out held exactly: half of that, the result's own rounding (of a number
        # that is at most half a step of X from exp), and those of two products and a sum in fp32
        most = 0.5 * HALF[dtype] * size + HALF[dtype] * (exp.abs() + 0.5 * HALF[dtype] * size) + 3 * 2.0 ** -24 * size
        assert ((out.double() - exp).abs() <= most).all()
        assert (wide[:, :5] == 7).all() and (wide[:, 75:] == 7).all() and (wide[..., 0] == 7).all() and (wide[..., 134:] == 7).all()
        H = G.to(dtype, copy=True)                    # (of the same type it would be G, which this changes)
        exp = s3r.orthogonalize(H)
        s3r.s3r_orthogonalize(H, H, ws=ws)
        assert torch.equal(H, exp)                    # in place
    nan = torch.full((5, 70, 133), float("nan"), dtype=torch.bfloat16, device=DEV)
    s3r.s3r_orthogonalize(G, nan, ws=ws)              # keep 0 reads nothing
    assert torch.equal(nan, each)
    tall = G.transpose(1, 2).contiguous()
    for e, y in enumerate(s3r.orthogonalize(tall)):
        check(y, tall[e])


def test_zeros_and_non_finite():
    G = gradient((4, 40, 50), torch.float32, 2)
    G[1] = 0
    G[2, 3, 4] = float("nan")
    G[3, 39, 49] = float("-inf")
    for eps in (0.0, 1e-7):
        y = s3r.orthogonalize(G, eps=eps)
        check(y[0], G[0], eps=eps)
        assert not y[1].any() and y[2:].isnan().all()
    low = gradient((40, 1), torch.float32, 4) @ gradient((1, 50), torch.float32, 5)       # rank one
    check(s3r.orthogonalize(low), low)
    for shape in ((0, 5), (5, 0), (0, 3, 4), (2, 0, 4)):
        assert s3r.orthogonalize(torch.empty(shape, device=DEV)).shape == shape


def exact64(G, steps=5):
    """The steps in float64 on the GPU, which torch's products do quickly enough for the large tiles."""
    a, b, c = (float(np.float32(v)) for v in orth.COEFFS)
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.t().contiguous() if tall else X
    X = X / (X.norm() + float(np.float32(1e-7)))
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.t() if tall else X


@pytest.mark.parametrize("shape", [(2048, 2048), (1500, 4000), (4000, 1500), (4096, 4096), (3900, 6000), (6200, 4097), (64, 60000)])
def test_large(shape):
    """Tiles of 128 and 256, shared among workgroups and not; errors as of the small ones."""
    g = torch.Generator(DEV).manual_seed(1)
    G = torch.randn(*shape, generator=g, device=DEV) * 1e-3
    G += torch.randn(shape[0], 1, generator=g, device=DEV) @ torch.randn(1, shape[1], generator=g, device=DEV) * 1e-2
    exp = exact64(G)
    y = s3r.orthogonalize(G)
    off = float((y.double() - exp).norm() / exp.norm())
    print(f"{shape}: {off:.2e}")
    # measured by the small matrices' rule: 2^-22 of the magnitudes at every step; the longest sums here add
    # 60000 terms, whose fp32 roundings may be 2^-25 sqrt(3 * 60000 / 16) = 2^-18 of them
    assert off <= 1e-5
    assert torch.equal(y, s3r.orthogonalize(G))


@pytest.mark.parametrize("shape", [(2, 1500, 2600), (3, 2600, 1100), (2, 2304, 4352)])
def test_several_large(shape):
    """Shared tiles of more than one matrix; results in bf16, whose last steps take one plane."""
    g = torch.Generator(DEV).manual_seed(3)
    G = torch.randn(*shape, generator=g, device=DEV)
    y, z = s3r.orthogonalize(G), s3r.orthogonalize(G, out_dtype=torch.bfloat16)
    for e in range(shape[0]):
        exp = exact64(G[e])
        assert float((y[e].double() - exp).norm() / exp.norm()) <= 1e-5
        # half a step of bf16, and as much again at most for what the last steps leave out
        assert float((z[e].double() - exp).norm() / exp.norm()) <= 2 * 2.0 ** -8


def test_smallest_values_are_kept():
    """X far below 1 (eps is most of the norm): to 2^-37 absolute, through planes whose values are subnormal fp16."""
    G = gradient((70, 90), torch.float32, 8, 1e-11)
    for steps in (1, 3):
        y = s3r.orthogonalize(G, steps=steps, coeffs=(1.0, 0.0, 0.0), eps=1e-2)
        exp = host(G.double()) / (np.linalg.norm(host(G.double())) + float(np.float32(1e-2)))
        off = np.abs(host(y.double()) - exp).max()
        print(f"{off:.2e}, values to {np.abs(exp).max():.2e}")
        assert off <= steps * 2.0 ** -37 + 2.0 ** -23 * np.abs(exp).max()


def test_many_matrices_in_tiles_of_128():
    G = gradient((20, 300, 700), torch.bfloat16, 9)
    y = s3r.orthogonalize(G, out_dtype=torch.float32)
    for e in (0, 7, 19):
        check(y[e], G[e])


def test_singular_values_near_one():
    g = torch.Generator(DEV).manual_seed(2)
    for shape in ((200, 300), (300, 200)):
        s = torch.linalg.svdvals(s3r.orthogonalize(torch.randn(*shape, generator=g, device=DEV)).double().cpu())
        assert 0.6 < float(s.min()) and float(s.max()) < 1.3


def test_streams_and_graph_replays():
    G = gradient((3, 200, 300), torch.float32, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y0 = s3r.orthogonalize(G, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y0, s3r.orthogonalize(G))
    out, ws = torch.empty_like(G), s3r.orthogonalize_buffer(G)
    long, long_out = gradient((64, 8192), torch.float32, 2), torch.empty(64, 8192, device=DEV)
    ws2 = s3r.orthogonalize_buffer(long)

    def step():
        s3r.s3r_orthogonalize(G, out, ws=ws)
        s3r.s3r_orthogonalize(long, long_out, ws=ws2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        G.copy_(gradient((3, 200, 300), torch.float32, 10 + seed))
        long.copy_(gradient((64, 8192), torch.float32, 20 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), long_out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], long_out)


def low_rank(shape, rank, seed=0, size=1e-4):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.normal(size=(shape[0], rank)) @ r.normal(size=(rank, shape[1])) * size).float().to(DEV)


def lost(shape, steps=5, a=orth.COEFFS[0]):
    """How far a result may be off where G has few directions, of its norm: (2^-22 + 2^-24 sqrt(n / 16)) a^steps, n the longer side.

    A value is kept to 2^-24 of itself and a product leaves out 2^-24 of its terms.  A sum of n terms of one sign is made by
    3 n / 16 additions to a running sum that grows evenly, each off by 2^-24 of it at most and 2^-24 / sqrt(3) in the mean, all
    together 2^-24 sqrt(n / 16) / sqrt(3).  What falls into a direction that G lacks is multiplied there by a in every later
    step, as A's errors are in their own: by sqrt((b + c)^2 + c^2) = 3.4 for singular values near 1, which is a.  The later steps' own
    errors are a, a^2, .. times smaller: 1 / (1 - 1 / a) = 1.41 altogether, and 1.41 / sqrt(3) < 1.  The result's norm
    is that of G's directions, whose values stay near 1.
    """
    return (2.0 ** -22 + 2.0 ** -24 * np.sqrt(max(shape) / 16)) * max(1.0, a) ** steps


def bf16_rounding(exp):
    """How far the nearest bf16 values of a matrix are from it."""
    return np.linalg.norm(host(torch.from_numpy(exp).bfloat16().double()) - exp)


@pytest.mark.parametrize("rank", [1, 4, 8, 64, None])
@pytest.mark.parametrize("shape", [(100, 90), (256, 512), (700, 300)])
def test_results_in_bf16_lose_their_rounding_only(shape, rank):
    """A value's distance from its nearest bf16 moves by no more than the value does: off by d before the rounding, the
    result is off by the exact result's own rounding and 2 d at most."""
    for steps, coeffs in ((5, orth.COEFFS), (1, orth.COEFFS), (2, orth.COEFFS), (3, (1.5, -0.5, 0.0)), (6, (1.875, -1.25, 0.375))):
        G = gradient(shape, torch.float32, 3) if rank is None else low_rank(shape, rank)
        exp = orth.newton_schulz(host(G.double()), steps=steps, coeffs=coeffs)
        for H in (G, G.t().contiguous()):
            y = s3r.orthogonalize(H, steps=steps, coeffs=coeffs, out_dtype=torch.bfloat16)
            y = host((y if H is G else y.t()).double())
            most = bf16_rounding(exp) + 2 * lost(shape, steps, coeffs[0]) * np.linalg.norm(exp)
            off = np.linalg.norm(y - exp)
            print(f"{shape} rank {rank}, {steps} steps: {off / np.linalg.norm(exp):.2e} of {most / np.linalg.norm(exp):.2e}")
            assert off <= most


def into(G, out_dtype):
    """The steps' result through a workspace of NaN (every plane's fp16, every sum): what is read has been written."""
    out, ws = torch.empty(G.shape, dtype=out_dtype, device=DEV), s3r.orthogonalize_buffer(G)
    s3r.s3r_orthogonalize(G, out, ws=ws.fill_(255))
    return out


@pytest.mark.parametrize("shape", [*SHAPES, (3, 70, 133), (5, 130, 50), (20, 300, 700), (2, 1500, 2600)])
def test_workspaces_that_hold_anything(shape):
    G = gradient(shape, torch.float32, 6)
    for out in BOTH:
        assert torch.equal(into(G, out), s3r.orthogonalize(G, out_dtype=out))


# tiles of 256 for both kinds of product (and sides that fill none), of 128 and 256 (padding of X that no product writes)
WIDEST = [(4090, 8190), (8190, 4090), (2, 2300, 8100), (5220, 6100), (6100, 5220)]


@pytest.mark.parametrize("shape", WIDEST)
def test_widest_tiles(shape):
    """Errors as of the other large matrices, and the result's own rounding in bf16 (twice the error at most beside it)."""
    g = torch.Generator(DEV).manual_seed(4)
    G = torch.randn(*shape, generator=g, device=DEV)
    y, z = into(G, torch.float32), into(G, torch.bfloat16)
    for e in range(shape[0] if len(shape) == 3 else 1):
        at = (lambda t: t[e]) if len(shape) == 3 else (lambda t: t)
        exp = exact64(at(G))
        n = float(exp.norm())
        off, off16 = float((at(y).double() - exp).norm()), float((at(z).double() - exp).norm())
        rounding = float((exp.bfloat16().double() - exp).norm())
        print(f"{shape}: {off / n:.2e}, bf16 {off16 / n:.2e} of {rounding / n:.2e}")
        assert off <= 1e-5 * n and off16 <= rounding + 2e-5 * n


@pytest.mark.parametrize("rank", [1, 8])
@pytest.mark.parametrize("shape", [(2048, 1408), (1500, 4000), (4090, 8190), (5220, 6100)])
def test_low_rank_in_large_tiles(shape, rank):
    """Rounding errors fill the directions that G leaves empty, and each step multiplies them by a."""
    g = torch.Generator(DEV).manual_seed(rank)
    G = torch.randn(shape[0], rank, generator=g, device=DEV) @ torch.randn(rank, shape[1], generator=g, device=DEV) * 1e-4
    exp = exact64(G)
    most = lost(shape) * float(exp.norm())
    off = float((into(G, torch.float32).double() - exp).norm())
    off16 = float((into(G, torch.bfloat16).double() - exp).norm())
    rounding = float((exp.bfloat16().double() - exp).norm())
    print(f"{shape} rank {rank}: {off / float(exp.norm()):.2e} of {lost(shape):.2e}, bf16 {off16 / float(exp.norm()):.2e} of {rounding / float(exp.norm()):.2e}")
    assert off <= most and off16 <= rounding + 2 * most


@pytest.mark.parametrize("rank", [1, 2, 8, 32, None])
@pytest.mark.parametrize("steps", [3, 5, 8, 10])
def test_errors_by_rank_and_steps(rank, steps):
    for shape in ((256, 512), (64, 90), (300, 129)):
        G = gradient(shape, torch.float32, steps) if rank is None else low_rank(shape, rank, steps)
        exp = orth.newton_schulz(host(G.double()), steps=steps)
        off = np.linalg.norm(host(s3r.orthogonalize(G, steps=steps).double()) - exp) / np.linalg.norm(exp)
        most = lost(shape, steps)
        print(f"{shape} rank {rank}, {steps} steps: {off:.2e} of {most:.2e}")
        assert off <= most


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("size", [1e-35, 1e-37, 1e-38, 1e-40, 2e37])
def test_norms_whose_inverse_leaves_fp32(size, dtype):
    """Without an eps every matrix is brought to norm 1, down to subnormal elements and up to the largest."""
    for shape in ((70, 90), (90, 70), (1, 1), (300, 700)):
        G = gradient(shape, dtype, 3, size)
        assert bool(G.isfinite().all()) and bool(G.any())
        check(s3r.orthogonalize(G, eps=0.0, out_dtype=torch.float32), G, eps=0.0)


@pytest.mark.parametrize("shape", [(1, (1 << 20) - 1), ((1 << 20) - 1, 3), (2, 5, 700001)])
def test_longest_sides(shape):
    G = gradient(shape, torch.float32, 7)
    y = into(G, torch.float32)
    for g, u in ((G, y),) if len(shape) == 2 else zip(G, y):
        exp = orth.newton_schulz(host(g.double()))
        assert np.linalg.norm(host(u.double()) - exp) <= lost(shape) * np.linalg.norm(exp)
