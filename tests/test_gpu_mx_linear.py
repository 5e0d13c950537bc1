"""MXFP4 rows and forward products on an MI355X against oracle/mx.py.

Codes and scales are equal.  A product of values that MXFP4 stands for is exact in fp32, so y carries only
the K additions: at most one rounding of 2^-23 (the matrix cores may truncate) of the running magnitude each,
K 2^-23 sum |a| |b|; a bf16 result adds half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import mx, swiglu
from stochastic_rounding_quantization_amd import s3r
from tests._gpu import DEV, host, mx_rows as plain_codes

pytestmark = pytest.mark.gpu


def matrix(shape, dtype, seed, outliers=True):
    r = np.random.default_rng(seed)
    x = r.normal(size=shape) * np.exp2(r.integers(-6, 6, shape[:-1] + (1,)))
    if outliers and x.size:
        x.reshape(-1)[r.integers(0, x.size, 1 + x.size // 200)] *= 300
    return torch.from_numpy(x).to(DEV, dtype)


def f32(t):
    return host(t.float())


def check_rows(q, exp, group=0):
    K = q.K
    steps = (K + 127) // 128
    np.testing.assert_array_equal(plain_codes(q.codes[group], q.rows, 128 * steps), mx.pack(exp["codes"]))
    scale = host(q.scales[group]).reshape(steps, q.rows, 4).transpose(1, 0, 2).reshape(q.rows, 4 * steps)
    np.testing.assert_array_equal(scale, exp["scale"])


def check_product(y, a, b):
    """a [M x K], b [N x K]: the values that MXFP4 stands for."""
    exp, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 0.0
    got = host(y.double())
    assert (np.abs(got - exp) <= (a.shape[1] + 4) * 2.0 ** -23 * mag + half * (1 + 1e-3) * np.abs(exp)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R, K", [(1, 1), (1, 128), (3, 31), (16, 96), (17, 300), (256, 64), (300, 1411), (513, 256)])
def test_rows(R, K, dtype):
    A = matrix((R, K), dtype, R + K)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    check_rows(s3r.mx_rows(A, flags=flags), mx.rows(f32(A)))
    assert int(flags) == 0


def test_rows_borders_and_non_finite():
    # every tie, both signs, the largest of each binade, zeros, subnormals
    vals = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 0.5, 1, 1.5, 2, 3, 4, 5.99, 2.49, 2.51, 0.249, 0.251], np.float32)
    row = np.concatenate([vals, -vals])[:32]
    rows = np.stack([row * 2.0 ** e for e in (-149, -140, -130, -127, -126, -3, 0, 5, 100, 124)]).astype(np.float32)
    rows = np.concatenate([rows, np.zeros((1, 32), np.float32), np.full((1, 32), np.finfo(np.float32).max, np.float32)])
    check_rows(s3r.mx_rows(torch.from_numpy(rows).to(DEV)), mx.rows(rows))
    bad = np.random.default_rng(1).normal(size=(5, 200)).astype(np.float32)
    bad[1, 40], bad[2, 199], bad[4, 0] = np.nan, np.inf, -np.inf
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = s3r.mx_rows(torch.from_numpy(bad).to(DEV), flags=flags)
    check_rows(q, mx.rows(bad))
    assert int(flags) == s3r.FLAG_NONFINITE
    w = s3r.mx_rows(matrix((40, 200), torch.float32, 2))
    y = host(s3r.mx_product(q, w))
    assert np.isnan(y[[1, 2, 4]]).all() and np.isfinite(y[[0, 3]]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_rows_of_every_width(dtype, offset):
    """Row ends at every place of a 16-byte word, with NaN around the rows; two rows also as the product rounds them."""
    for K in [*range(1, 26), *range(120, 138), 255, 257]:
        wide = torch.full((22, K + 21), float("nan"), dtype=dtype, device=DEV)
        A = wide[1:21, offset:offset + K]
        A.copy_(matrix((20, K), dtype, K))
        check_rows(s3r.mx_rows(A), mx.rows(f32(A)))
        W = matrix((40, K), dtype, 7)
        y = s3r.mx_linear(A[:2], s3r.mx_rows(W), out_dtype=torch.float32)
        check_product(y, mx.rows(f32(A[:2]))["deq"], mx.rows(f32(W))["deq"])


def test_rows_strides_index_and_groups():
    wide = matrix((50, 400), torch.bfloat16, 3)
    for A in (wide[:, 1:301], wide[:, 8:308], wide[::3, :96]):
        check_rows(s3r.mx_rows(A), mx.rows(f32(A)))
    idx = torch.tensor([3, 99, 0, 100, -1, 55, 98], dtype=torch.int32, device=DEV)       # 100 // 2 is row 50: none
    exp = f32(wide)[[1, 49, 0, 0, 0, 27, 49]].copy()
    exp[3:5] = 0
    check_rows(s3r.mx_rows(wide, index=idx, index_div=2), mx.rows(exp))
    W = matrix((3, 70, 130), torch.bfloat16, 4)
    q = s3r.mx_rows(W)
    for g in range(3):
        check_rows(q, mx.rows(f32(W[g])), g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_silu_times_up(dtype):
    g, u = matrix((33, 300), dtype, 5), matrix((33, 300), dtype, 6)
    a, b = f32(g), f32(u)
    F = np.float32
    with np.errstate(all="ignore"):
        s = (F(1) / (F(1) + swiglu.exp32(-a))).astype(F)
        h = ((a * s).astype(F) * b).astype(F)
    check_rows(s3r.mx_rows(g, up=u), mx.rows(h))


SHAPES = [(1, 1, 1), (1, 14, 128), (2, 100, 2048), (5, 33, 300), (16, 256, 640), (17, 130, 96), (40, 300, 1000),
          (64, 1411, 512), (129, 257, 384), (300, 513, 2024), (513, 128, 130), (260, 1000, 4096),
          (2, 70, 40000), (31, 9000, 96), (400, 3130, 130), (700, 4100, 200), (1500, 4100, 96), (3000, 4100, 129)]


@pytest.mark.parametrize("dtype, out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_linear(M, N, K, dtype, out):
    A, W = matrix((M, K), dtype, M + N), matrix((N, K), torch.bfloat16, N + K)
    w = s3r.mx_rows(W)
    y = s3r.mx_linear(A, w, out_dtype=out)
    a, b = mx.rows(f32(A))["deq"], mx.rows(f32(W))["deq"]
    check_product(y, a, b)
    y2 = s3r.mx_product(s3r.mx_rows(A), w, out_dtype=out)
    check_product(y2, a, b)
    assert torch.equal(s3r.mx_linear(A, w, out_dtype=out), y)               # the same bits again


def test_linear_writes_its_rows_and_columns_only():
    A, w = matrix((70, 256), torch.bfloat16, 7), s3r.mx_rows(matrix((90, 256), torch.bfloat16, 8))
    for dt in (torch.float32, torch.bfloat16):
        for rows in (3, 70):
            big = torch.full((72, 101), 5.0, dtype=dt, device=DEV)
            s3r.s3r_mx_linear(A[:rows], w, big[1:1 + rows, 3:93], ws=s3r.mx_linear_buffer(rows, 256, DEV))
            assert torch.equal(big[1:1 + rows, 3:93], s3r.mx_linear(A[:rows], w, out_dtype=dt))
            assert (big[0] == 5).all() and (big[1 + rows:] == 5).all() and (big[:, :3] == 5).all() and (big[:, 93:] == 5).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M, K", [(5, 200), (300, 129), (1500, 96)])
def test_linear_into_any_alignment(M, K, out):
    """Results of every width mod 16 bytes, from any element on, have an aligned result's bits; nothing else is written."""
    A = s3r.mx_rows(matrix((M, K), torch.bfloat16, M))
    W = matrix((2064, K), torch.bfloat16, K)
    for N in (1, 7, 65, 130, 1411, *range(2056, 2065)):
        w = s3r.mx_rows(W[:N])
        exp = s3r.mx_product(A, w, out_dtype=out)
        for offset in (0, 1, 2, 3, 8):
            wide = torch.full((M + 2, N + 17), 9.0, dtype=out, device=DEV)
            y = wide[1:M + 1, offset:offset + N]
            s3r.s3r_mx_product(A, w, y)
            assert torch.equal(y, exp)
            y.fill_(9)
            assert (wide == 9).all()


def test_empty_products():
    w = s3r.mx_rows(matrix((20, 64), torch.bfloat16, 9))
    assert s3r.mx_linear(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), w).shape == (0, 20)
    z = s3r.mx_rows_buffer(20, 0, DEV)
    for rows in (3, 24, 100):                                              # K = 0: an empty sum
        y = torch.full((rows, 20), 7.0, device=DEV)
        s3r.s3r_mx_product(s3r.mx_rows_buffer(rows, 0, DEV), z, y)
        assert (y == 0).all()


@pytest.mark.parametrize("rows", [1, 2, 5, 40, 200])
def test_non_finite_rows_and_indices_outside(rows):
    """A non-finite element makes its row NaN, an index outside the source makes its row zero, whichever kernel runs."""
    A, w = matrix((rows, 300), torch.bfloat16, 3), s3r.mx_rows(matrix((70, 300), torch.bfloat16, 4))
    idx = torch.arange(rows, dtype=torch.int32, device=DEV)
    want = s3r.mx_linear(A, w)
    A[rows // 2, 299] = float("inf")
    idx[0] = rows if rows > 1 else -1
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = s3r.mx_linear(A, w, flags=flags)
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[rows // 2] = True
    assert int(flags) == s3r.FLAG_NONFINITE and got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])
    got = s3r.mx_linear(A, w, index=idx)
    assert (got[0] == 0).all() and torch.equal(got[1:][~bad[1:]], want[1:][~bad[1:]])


def test_helpers_on_a_stream():
    A, w = matrix((300, 256), torch.bfloat16, 5), s3r.mx_rows(matrix((200, 256), torch.bfloat16, 6))
    want = s3r.mx_linear(A, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(10):                             # the workspaces of these overlap work of the current stream
        got.append(s3r.mx_linear(A, w, stream=side.cuda_stream))
        torch.zeros(1 << 20, device=DEV)
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


GROUPS = [([0, 1], 64, 96), ([5], 40, 128), ([1, 0, 2, 0, 0, 1], 100, 256), ([0, 0, 33, 16, 17], 70, 300),
          ([300, 0, 1, 129, 255, 256, 7], 150, 640), ([1] * 70, 33, 128), ([40] * 9, 257, 384), ([0, 700, 0], 130, 200),
          ([9, 3, 20, 30], 70, 200), ([2600, 0, 700], 300, 130)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts, N, K", GROUPS)
def test_grouped(counts, N, K, out):
    R, G = sum(counts), len(counts)
    T = R // 2 + 1
    X, W = matrix((T, K), torch.bfloat16, R), matrix((G, N, K), torch.bfloat16, G)
    idx = torch.from_numpy(np.random.default_rng(R).integers(0, 2 * T, R).astype(np.int32)).to(DEV)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)).to(DEV)
    w = s3r.mx_rows(W)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = s3r.mx_linear(X, w, offsets=off, index=idx, index_div=2, out_dtype=out, flags=flags)
    a = mx.rows(f32(X))["deq"][host(idx) // 2]
    o = host(off)
    for g in range(G):
        if o[g + 1] > o[g]:
            check_product(y[o[g]:o[g + 1]], a[o[g]:o[g + 1]], mx.rows(f32(W[g]))["deq"])
    assert int(flags) == 0


@pytest.mark.parametrize("R", [4, 8, 400, 8000])
def test_bad_offsets_compute_nothing(R):
    w = s3r.mx_rows(matrix((4, 64, 128), torch.bfloat16, 1))
    X = matrix((R, 128), torch.bfloat16, 2)
    for off in ([0, 3, 2, 4, R], [1, 2, 3, 4, R], [0, 1, 2, 3, R - 1], [0, 1, 2, R + 1, R], [0, -1, 2, 3, R],
                [0, 1, 1 << 40, 3, R]):
        y = torch.full((R, 64), 7.0, device=DEV)
        flags = torch.zeros(1, dtype=torch.int32, device=DEV)
        s3r.s3r_mx_linear(X, w, y, offsets=torch.tensor(off, device=DEV), ws=s3r.mx_linear_buffer(R, 128, DEV), flags=flags)
        assert (y == 7).all() and int(flags) == s3r.FLAG_BAD_GROUPS


def test_stream_and_graph_replays():
    X, w = matrix((200, 256), torch.bfloat16, 1), s3r.mx_rows(matrix((3, 90, 256), torch.bfloat16, 2))
    off = torch.tensor([0, 50, 50, 200], device=DEV)
    y, ws = torch.empty(200, 90, device=DEV), s3r.mx_linear_buffer(200, 256, DEV)
    one, y1 = s3r.mx_rows(matrix((1, 64, 256), torch.bfloat16, 3)), torch.empty(2, 64, device=DEV)
    ws1 = s3r.mx_linear_buffer(2, 256, DEV)

    def step():
        s3r.s3r_mx_linear(X, w, y, offsets=off, ws=ws)
        s3r.s3r_mx_linear(X[:2], one, y1, ws=ws1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        X.copy_(matrix((200, 256), torch.bfloat16, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), y1.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], y1)


def test_bf16_rows_borders_and_non_finite():
    """As test_rows_borders_and_non_finite in bf16, which has its own maximum and conversion: from its smallest subnormal."""
    vals = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 0.5, 1, 1.5, 2, 3, 4, 5.96875, 2.484375, 2.515625, 0.2490234375,
                     0.2509765625], np.float32)                              # exact in bf16 but for the smallest exponents
    row = np.concatenate([vals, -vals])[:32]
    rows = np.stack([row * 2.0 ** e for e in (-133, -132, -131, -130, -129, -128, -127, -126, -125, -3, 0, 5, 100, 125)])
    most = float(torch.finfo(torch.bfloat16).max)
    rows = np.concatenate([rows, np.zeros((1, 32)), -np.zeros((1, 32)), np.full((1, 32), most), np.full((1, 32), -most)])
    rows = np.concatenate([rows, np.eye(4, 32) * 2.0 ** -133, np.eye(4, 32) * -(2.0 ** -126)])
    A = torch.from_numpy(rows.astype(np.float32)).to(DEV).bfloat16()
    check_rows(s3r.mx_rows(A), mx.rows(f32(A)))
    w = s3r.mx_rows(matrix((40, 32), torch.bfloat16, 3))
    for i in range(0, len(rows), 2):                     # rounded by the product itself
        assert torch.equal(s3r.mx_linear(A[i:i + 2], w, out_dtype=torch.float32),
                           s3r.mx_product(s3r.mx_rows(A[i:i + 2]), w))
    bad = torch.from_numpy(np.random.default_rng(1).normal(size=(5, 200)).astype(np.float32)).to(DEV).bfloat16()
    bad[1, 40], bad[2, 199], bad[4, 0] = float("nan"), float("inf"), float("-inf")
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = s3r.mx_rows(bad, flags=flags)
    check_rows(q, mx.rows(f32(bad)))
    assert int(flags) == s3r.FLAG_NONFINITE
    y = host(s3r.mx_product(q, s3r.mx_rows(matrix((40, 200), torch.bfloat16, 2))))
    assert np.isnan(y[[1, 2, 4]]).all() and np.isfinite(y[[0, 3]]).all()


def test_no_rows_gathered():
    X, w = matrix((9, 64), torch.bfloat16, 1), s3r.mx_rows(matrix((3, 20, 64), torch.bfloat16, 2))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert s3r.mx_rows(X, index=none, index_div=2).rows == 0
    y = s3r.mx_linear(X, w, offsets=torch.zeros(4, dtype=torch.int64, device=DEV), index=none, index_div=2)
    assert y.shape == (0, 20)


@pytest.mark.parametrize("R, N", [(0, 20), (5, 0), (0, 0)])
def test_offsets_of_an_empty_product(R, N):
    """They are looked at as those of any product."""
    bf16 = dict(dtype=torch.bfloat16, device=DEV)
    w, a = s3r.mx_rows(torch.ones(70, N, 64, **bf16)), torch.ones(R, 64, **bf16)
    y, ws = torch.empty(R, N, device=DEV), s3r.mx_linear_buffer(R, 64, DEV)
    good = torch.full((71,), R, dtype=torch.int64, device=DEV)
    good[:30] = 0
    for at, value in ((None, 0), (0, 1), (70, R + 1), (65, R + 1), (3, -1)):
        off = good.clone()
        if at is not None:
            off[at] = value
        for flags in (None, torch.zeros(2, dtype=torch.int32, device=DEV)):
            f = None if flags is None else flags[:1]
            s3r.s3r_mx_product(s3r.mx_rows(a), w, y, offsets=off, flags=f)
            s3r.s3r_mx_linear(a, w, y, offsets=off, ws=ws, flags=None if flags is None else flags[1:])
            if flags is not None:
                assert host(flags).tolist() == ([0, 0] if at is None else [s3r.FLAG_BAD_GROUPS] * 2)
