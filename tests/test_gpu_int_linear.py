"""INT8 rows, their column sums and forward products on an MI355X against oracle/int8.py.

Sums are integers and every other operation is one fp32 rounding in a stated order, so everything is equal, bit for bit:
codes, steps, and results by each of the products' kernels.
"""
import numpy as np
import pytest
import torch

from oracle import int8
from stochastic_rounding_quantization_amd import s3r
from tests._gpu import DEV, host

pytestmark = pytest.mark.gpu
BOTH = [torch.float32, torch.bfloat16]


def matrix(shape, dtype, seed):
    """Rows of very different sizes, with outliers."""
    r = np.random.default_rng(seed)
    x = r.normal(size=shape) * np.exp2(r.integers(-6, 6, shape[:-1] + (1,)))
    if x.size:
        x.reshape(-1)[r.integers(0, x.size, 1 + x.size // 200)] *= 30
    return torch.from_numpy(x).to(DEV, dtype)


def f32(t):
    return host(t.float())


def check_rows(q, exp, group=0):
    codes, delta, _ = exp
    np.testing.assert_array_equal(host(q.codes[group])[:, :q.K], codes)
    assert not host(q.codes[group])[:, q.K:].any()
    np.testing.assert_array_equal(host(q.delta[group]), delta)


def same(y, exp):
    """Equal, NaN where NaN."""
    np.testing.assert_array_equal(f32(y), exp)


def expected(x, w, bias=None, up=None, out=torch.float32, group=0):
    qa, sa, _ = int8.rows(f32(x), None if up is None else f32(up))
    return int8.product(qa, sa, host(w.Q if w.groups == 1 else w.Q[group]), host(w.delta[group]),
                        None if bias is None else f32(bias), out is torch.bfloat16)


LENGTHS = [1, 7, 8, 15, 16, 17, 100, 511, 513, 2047, 2048, 2049, 4096, 4097, 8192, 8193, 14336, 16384, 16385, 40000]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", LENGTHS)
def test_rows(K, dtype):
    A = matrix((5, K), dtype, K)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = s3r.int_rows(A, flags=flags)
    check_rows(q, int8.rows(f32(A)))
    f = s3r.forward_operand(A)
    assert torch.equal(f.Q, q.Q) and torch.equal(f.delta, q.delta[0]) and int(flags) == 0


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", [1, 9, 300, 2050, 5001, 17000])
def test_rows_of_gate_and_up(K, dtype):
    both = matrix((7, 2 * K), dtype, K) * 0.1
    gate, up = both[:, :K], both[:, K:]
    check_rows(s3r.int_rows(gate, up=up), int8.rows(f32(gate), f32(up)))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_rows_of_every_width(dtype, offset):
    """Row ends at every place of a 16-byte word, with NaN around the rows; two rows also as the product rounds them."""
    for K in [*range(1, 26), *range(120, 138), 1023, 1025]:
        wide = torch.full((22, K + 21), float("nan"), dtype=dtype, device=DEV)
        A = wide[1:21, offset:offset + K]
        A.copy_(matrix((20, K), dtype, K))
        q = s3r.int_rows(A)
        check_rows(q, int8.rows(f32(A)))
        w = s3r.int_rows(matrix((5, K), dtype, K + 1))
        for n in (1, 2, 4):
            same(s3r.int_linear(A[:n], w, out_dtype=torch.float32), expected(A[:n], w))


@pytest.mark.parametrize("dtype", BOTH)
def test_borders_zeros_and_non_finite(dtype):
    vals = np.array([127, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5, 0, 1, -127, 63.5, 0.49, 0.51, -0.0, 3], np.float32)
    rows = np.stack([vals * 2.0 ** e for e in (-100, -20, 0, 1, 60)] + [vals * 0, vals * 2.0 ** -140, vals * 1e-30])
    A = torch.from_numpy(rows.astype(np.float32)).to(DEV, dtype)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = s3r.int_rows(A, flags=flags)
    exp = int8.rows(f32(A))
    check_rows(q, exp)
    assert int(flags) == exp[2] == s3r.FLAG_TINY_STEP
    bad = matrix((6, 700), dtype, 3)
    bad[1, 40], bad[2, 699], bad[4, 0] = float("nan"), float("inf"), float("-inf")
    w = s3r.int_rows(matrix((40, 700), dtype, 2))
    flags.zero_()
    q = s3r.int_rows(bad, flags=flags)
    check_rows(q, int8.rows(f32(bad)))
    assert int(flags) == s3r.FLAG_NONFINITE
    y = s3r.int_product(q, w)
    same(y, expected(bad, w))
    assert np.isnan(f32(y)[[1, 2, 4]]).all() and np.isfinite(f32(y)[[0, 3, 5]]).all()
    for n in (1, 2, 3):                           # rounded by the product itself
        flags.zero_()
        y = s3r.int_linear(bad[:n], w, flags=flags, out_dtype=torch.float32)
        same(y, expected(bad[:n], w))
        assert int(flags) == (s3r.FLAG_NONFINITE if n > 1 else 0)


def test_rows_gathered_and_of_several_matrices():
    X = matrix((9, 333), torch.bfloat16, 5)
    index = torch.tensor([4, 0, 17, 18, -1, 2, 2, 1 << 30], dtype=torch.int32, device=DEV)
    src = host(X.float())[[2, 0, 8, 0, 0, 1, 1, 0]]
    src[[3, 4, 7]] = 0
    check_rows(s3r.int_rows(X, index=index, index_div=2), int8.rows(src))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert s3r.int_rows(X, index=none).rows == 0
    W = matrix((3, 50, 101), torch.float32, 6)
    q = s3r.int_rows(W)
    for e in range(3):
        check_rows(q, int8.rows(f32(W[e])), e)
    spaced = torch.empty(3, 60, 120, device=DEV)[:, 3:53, 5:106]
    spaced.copy_(W)
    p = s3r.int_rows(spaced)
    assert torch.equal(p.codes, q.codes) and torch.equal(p.delta, q.delta)


# every kernel: byte dot products (to 4 rows), few rows (to 64), each tile
SIZES = [(1, 1, 1), (1, 130, 1024), (1, 4099, 300), (2, 37, 5000), (3, 64, 65), (4, 1000, 14336), (4, 33, 15000),
         (5, 7, 3), (16, 100, 127), (17, 33, 129), (32, 257, 2100), (33, 16, 64), (64, 65, 1000), (65, 3, 31),
         (100, 130, 200), (130, 700, 333), (300, 1283, 128), (517, 1411, 1999), (1000, 3000, 257), (700, 9000, 96),
         (2100, 6200, 130), (4090, 3585, 1), (4096, 3584, 256)]


@pytest.mark.parametrize("out", BOTH)
@pytest.mark.parametrize("M, N, K", SIZES)
def test_products(M, N, K, out):
    x, W = matrix((M, K), torch.bfloat16, M + K), matrix((N, K), torch.bfloat16, N)
    w = s3r.int_rows(W)
    a = s3r.int_rows(x)
    a.codes[..., K:] = 77                         # columns past K may hold anything
    w.codes[..., K:] = -99
    bias = matrix((1, N), torch.float32, 7)[0] if (M + N) % 2 else None
    exp = expected(x, w, bias, out=out)
    wide = torch.full((M + 2, N + 3), 5.0, dtype=out, device=DEV)
    s3r.s3r_int_product(a, w, wide[1:-1, 1:-2], bias=bias)
    same(wide[1:-1, 1:-2], exp)
    assert (wide[0] == 5).all() and (wide[-1] == 5).all() and (wide[:, 0] == 5).all() and (wide[:, -2:] == 5).all()
    same(s3r.int_linear(x, w, bias=bias, out_dtype=out), exp)


@pytest.mark.parametrize("M, N, K", [(1, 300, 14336), (2, 65, 100), (4, 64, 9000), (7, 50, 700), (90, 200, 513)])
def test_gate_and_up_products(M, N, K):
    both = matrix((M, 2 * K), torch.bfloat16, K) * 0.1
    w = s3r.int_rows(matrix((N, K), torch.bfloat16, N))
    gate, up = both[:, :K], both[:, K:]
    same(s3r.int_linear(gate, w, up=up), expected(gate, w, up=up, out=torch.bfloat16))


def test_largest_sums():
    """All codes 127 (or of opposite signs) over the longest K: 2114060288 has to fit."""
    K = 131072
    w = s3r.int_rows(torch.ones(40, K, device=DEV))
    for M in (1, 4, 5, 20, 70):
        x = torch.ones(M, K, device=DEV)
        x[1::2] = -1
        a = s3r.int_rows(x)
        assert (a.codes[0, 0] == 127).all()
        same(s3r.int_product(a, w), expected(x, w))


def test_no_contraction_and_no_rows():
    w = s3r.int_rows(torch.empty(6, 0, device=DEV))
    assert (w.delta == 1).all()
    bias = torch.arange(6.0, device=DEV)
    for M in (1, 3, 9, 100):
        x = torch.empty(M, 0, device=DEV)
        assert torch.equal(s3r.int_linear(x, w, bias=bias), bias.expand(M, 6))
        assert not s3r.int_product(s3r.int_rows(x), w).any()
    w = s3r.int_rows(matrix((6, 20), torch.float32, 1))
    assert s3r.int_linear(torch.empty(0, 20, device=DEV), w).shape == (0, 6)


def grouped(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int64, device=DEV)


GROUPS = [[1, 0, 0, 3, 1], [0, 0, 5], [0] * 70 + [1, 2] + [0] * 60 + [1], [2, 9, 0, 17, 33, 1], [40, 0, 129, 3, 300],
          [1500, 0, 700, 2000], [5000], [0, 1]]


@pytest.mark.parametrize("K", [64, 1100])
@pytest.mark.parametrize("sizes", GROUPS, ids=[str(sum(g)) + "rows" for g in GROUPS])
def test_groups(sizes, K):
    E, N, R = len(sizes), 131, sum(sizes)
    offsets = grouped(sizes)
    x = matrix((R, K), torch.bfloat16, R)
    w = s3r.int_rows(matrix((E, N, K), torch.bfloat16, E))
    bias = matrix((E, N), torch.float32, 3)
    exp = np.concatenate([expected(x[a:b], w, bias[e], group=e)
                          for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:]))])
    same(s3r.int_linear(x, w, offsets=offsets, bias=bias, out_dtype=torch.float32), exp)
    a = s3r.int_rows(x)
    a.codes[..., K:] = 1
    same(s3r.int_product(a, w, offsets=offsets, bias=bias), exp)
    # gathered: two rows a token
    perm = torch.randperm(R, device=DEV).to(torch.int32)
    tokens = matrix(((R + 1) // 2, K), torch.bfloat16, R + 1)
    got = s3r.int_linear(tokens, w, offsets=offsets, index=perm, index_div=2, out_dtype=torch.float32)
    assert torch.equal(got, s3r.int_linear(tokens[perm.long() // 2].contiguous(), w, offsets=offsets, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [1, 2, 4, 9, 40, 100, 300])
def test_dense_gathers(M):
    """An index without groups, with places that name no row (zeros: the bias alone), and behind silu(gate) * up."""
    X = matrix((37, 500), torch.bfloat16, M) * 0.1
    w = s3r.int_rows(matrix((70, 250), torch.bfloat16, 3))
    bias = matrix((1, 70), torch.float32, 4)[0]
    index = torch.randint(0, 111, (M,), device=DEV).to(torch.int32)
    index[M // 2] = -5
    index[M // 3] = 111
    src = X[(index.long() // 3).clamp(0, 36)].clone()
    src[[M // 2, M // 3]] = 0
    gate, up = X[:, :250], X[:, 250:]
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = s3r.int_linear(gate, w, index=index, index_div=3, bias=bias, out_dtype=torch.float32, flags=flags)
    same(y, expected(src[:, :250], w, bias))
    assert torch.equal(y[M // 2], bias) and int(flags) == 0
    same(s3r.int_linear(gate, w, up=up, index=index, index_div=3, out_dtype=torch.float32),
         expected(src[:, :250], w, up=src[:, 250:]))


@pytest.mark.parametrize("M", [1, 3, 4])
def test_longest_rows_of_the_byte_products(M):
    """Rows past the registers of their workgroup, and past its LDS."""
    for K in (16384 // (4 if M > 2 else M), 4097, 13000, 15001, 17000, 59000, 60001):
        for dtype in BOTH:
            both = matrix((M, 2 * K), dtype, K) * 0.1
            w = s3r.int_rows(matrix((9, K), torch.bfloat16, 1))
            same(s3r.int_linear(both[:, :K], w, out_dtype=torch.float32), expected(both[:, :K], w))
            same(s3r.int_linear(both[:, :K], w, up=both[:, K:], out_dtype=torch.float32), expected(both[:, :K], w, up=both[:, K:]))


def test_groups_refuse_bad_offsets():
    w = s3r.int_rows(matrix((70, 20, 64), torch.bfloat16, 1))
    for R in (5, 70, 2000, 90000):
        x = torch.ones(R, 64, dtype=torch.bfloat16, device=DEV)
        good = torch.full((71,), R, dtype=torch.int64, device=DEV)
        good[:30] = 0
        for at, value in ((0, 1), (70, R + 1), (65, R + 1), (3, -1), (69, R - 1), (70, R - 1)):
            off = good.clone()
            off[at] = value
            ok = bool((off.diff() >= 0).all() and off[0] == 0 and off[-1] == R)
            flags = torch.zeros(3, dtype=torch.int32, device=DEV)
            y = torch.full((R, 20), 3.0, device=DEV)
            s3r.s3r_int_product(s3r.int_rows(x), w, y, offsets=off, flags=flags[:1])
            s3r.s3r_int_linear(x, w, y, offsets=off, flags=flags[1:2], ws=s3r.int_linear_buffer(R, 64, DEV))
            sums = torch.full((70, 64), 3, dtype=torch.int32, device=DEV)
            s3r.s3r_int_colsum(s3r.int_rows(x).Q, sums, offsets=off, flags=flags[2:])
            assert host(flags).tolist() == [0 if ok else s3r.FLAG_BAD_GROUPS] * 3
            assert ok or ((y == 3).all() and (sums == 3).all())
            s3r.s3r_int_linear(x, w, y, offsets=off, ws=s3r.int_linear_buffer(R, 64, DEV))


@pytest.mark.parametrize("R, K", [(0, 5), (1, 1), (64, 1024), (65, 1025), (1000, 333), (4096, 4096)])
def test_column_sums(R, K):
    A = matrix((R, K), torch.bfloat16, R + 1)
    q = s3r.int_rows(A)
    q.codes[..., K:] = 55
    assert torch.equal(s3r.int_colsum(q.Q), q.Q.sum(0, dtype=torch.int32)[None])
    if R and R % 4 == 0:
        assert torch.equal(s3r.int_colsum(q.Q, 4), q.Q.reshape(4, R // 4, K).sum(1, dtype=torch.int32))
    rng = np.random.default_rng(R)
    for G in (1, 3, 130):
        cuts = np.sort(rng.integers(0, R + 1, G - 1))
        off = torch.tensor(np.concatenate([[0], cuts, [R]]), dtype=torch.int64, device=DEV)
        o = off.tolist()
        exp = torch.stack([q.Q[a:b].sum(0, dtype=torch.int32) for a, b in zip(o, o[1:])])
        assert torch.equal(s3r.int_colsum(q.Q, offsets=off), exp)


def exact_rows(a, w, rows, group=0, first=0):
    """Results of single rows in float64."""
    return (a.Q[rows].double() @ w.codes[group, :, :w.K].double().t()) * (a.delta[0, rows, None].double() * w.delta[group].double())


def test_codes_past_32_bits():
    """Weights of 4.8 GB, rows of 5.4 GB: offsets of both operands and of the results pass 2^32."""
    E, N, K = 8, 30000, 20000
    w = s3r.IntRows(torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device=DEV), torch.rand(E, N, device=DEV), N, K, E)
    for R in (8, 160):                       # byte dot products or few rows, and tiles
        offsets = torch.arange(E + 1, device=DEV) * (R // E)
        x = matrix((R, K), torch.bfloat16, 1)
        y = s3r.int_linear(x, w, offsets=offsets, out_dtype=torch.float32)
        last = slice(R - R // E, R)
        exp = exact_rows(s3r.int_rows(x), w, last, E - 1)
        assert torch.allclose(y[last].double(), exp, rtol=2.0 ** -22, atol=0)
    del w
    R, K, N = 41000, 131072, 20
    a = s3r.IntRows(torch.randint(-127, 128, (1, R, K), dtype=torch.int8, device=DEV), torch.rand(1, R, device=DEV), R, K)
    w = s3r.int_rows(matrix((N, K), torch.bfloat16, 2))
    y = s3r.int_product(a, w)
    rows = slice(R - 100, R)
    assert torch.allclose(y[rows].double(), exact_rows(a, w, rows), rtol=2.0 ** -22, atol=0)
    assert torch.equal(s3r.int_colsum(a.Q[:, 130992:], 41)[40], a.Q[40000:, 130992:].sum(0, dtype=torch.int32))


def test_streams_and_graph_replays():
    X = matrix((200, 300), torch.bfloat16, 1)
    w = s3r.int_rows(matrix((70, 300), torch.bfloat16, 2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y0 = s3r.int_linear(X, w, stream=side.cuda_stream)
    c0 = s3r.int_colsum(s3r.int_rows(X, stream=side.cuda_stream).Q, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y0, s3r.int_linear(X, w)) and torch.equal(c0, s3r.int_colsum(s3r.int_rows(X).Q))
    outs = [torch.empty(n, 70, dtype=torch.bfloat16, device=DEV) for n in (200, 3, 30)]
    bufs = [s3r.int_linear_buffer(n, 300, DEV) for n in (200, 3, 30)]
    q, sums = s3r.int_rows_buffer(200, 300, DEV), torch.empty(2, 300, dtype=torch.int32, device=DEV)

    def step():
        for y, ws in zip(outs, bufs):
            s3r.s3r_int_linear(X[:y.shape[0]], w, y, ws=ws)
        s3r.s3r_int_rows(X, q)
        s3r.s3r_int_colsum(q.Q, sums)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        X.copy_(matrix((200, 300), torch.bfloat16, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*outs, sums)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*outs, sums)))


# few rows of wide weights (to 16, 32 and 64 rows) on both sides of 4096 columns, and tiles of 128 x 64
WIDE = [(7, 4096, 200), (16, 4097, 130), (20, 4090, 300), (30, 5000, 77), (60, 4095, 128), (40, 4100, 1000),
        (5, 8195, 300), (9, 8192, 64), (16, 14336, 129), (24, 8192, 1000), (32, 8449, 127), (33, 8200, 129), (50, 9001, 700),
        (64, 14336, 260), (512, 3100, 200), (500, 3333, 1029)]


@pytest.mark.parametrize("out", BOTH)
@pytest.mark.parametrize("M, N, K", WIDE)
def test_wide_products(M, N, K, out):
    test_products(M, N, K, out)


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", [256, 2043])
@pytest.mark.parametrize("N", [9, 8200])
def test_byte_products_of_every_kind(N, K, dtype, up):
    """One and four weight rows a wave; dense and over experts; rows rounded by the product itself and before it."""
    def both(rows, seed):
        x = matrix((rows, 2 * K), dtype, seed) * 0.1
        return (x[:, :K].contiguous(), x[:, K:].contiguous()) if up else (x[:, :K].contiguous(), None)

    def results(x, u, w, **kw):
        yield s3r.int_linear(x, w, up=u, out_dtype=torch.float32, **kw)
        yield s3r.int_product(s3r.int_rows(x, up=u), w, **kw)
    w = s3r.int_rows(matrix((N, K), torch.bfloat16, N))
    for M in (1, 2, 3, 4):
        x, u = both(M, M)
        exp = expected(x, w, up=u)
        for y in results(x, u, w):
            same(y, exp)
        same(s3r.int_linear(x, w, up=u, out_dtype=torch.bfloat16), expected(x, w, up=u, out=torch.bfloat16))
    sizes = [2, 0, 1, 0, 1]
    E, R, offsets = len(sizes), sum(sizes), grouped(sizes)
    N = min(N, 1700)                                # four rows a wave from here on, with the groups' five row tiles
    w = s3r.int_rows(matrix((E, N, K), torch.bfloat16, N + 1))
    x, u = both(R, 9)
    o = offsets.tolist()
    exp = np.concatenate([expected(x[a:b], w, up=None if u is None else u[a:b], group=e) for e, (a, b) in enumerate(zip(o, o[1:]))])
    for y in results(x, u, w, offsets=offsets):
        same(y, exp)


def random_rows(rows, K, groups=1):
    """Codes and steps without the rows behind them."""
    w = s3r.int_rows_buffer(rows, K, DEV, groups)
    w.codes.random_(-127, 128)
    w.delta.uniform_(0.5, 1.0)
    return w


def part(a, w, rows, cols, e=0):
    """Results of a slice of rows and columns: sums of 16 products are exact in fp32."""
    acc = a.Q[rows].float() @ w.codes[e, cols, :w.K].float().t()
    return (a.delta[0, rows, None] * w.delta[e, None, cols]) * acc


# more workgroups than a grid of one dimension has threads for
@pytest.mark.parametrize("M, N, out", [(2, (1 << 28) + 5, torch.float32), (9, (1 << 29) + 3, torch.bfloat16)])
def test_products_of_very_many_columns(M, N, out):
    a, w = random_rows(M, 16), random_rows(N, 16)
    y = torch.full((M, N), float("nan"), dtype=out, device=DEV)
    s3r.s3r_int_product(a, w, y)
    for cols in (slice(0, 1 << 22), slice(N // 2, N // 2 + (1 << 22)), slice(N - (1 << 22), N)):
        assert torch.equal(y[:, cols], part(a, w, slice(None), cols).to(out))
    assert not any(y[:, c:c + (1 << 27)].isnan().any() for c in range(0, N, 1 << 27))


def test_products_of_gate_and_up_with_very_many_columns():
    M, N = 2, (1 << 28) + 5
    w = random_rows(N, 16)
    both = matrix((M, 32), torch.bfloat16, 1)
    gate, up = both[:, :16], both[:, 16:]
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    s3r.s3r_int_linear(gate, w, y, up=up, ws=s3r.int_linear_buffer(M, 16, DEV))
    a = s3r.int_rows(gate, up=up)
    for cols in (slice(0, 1 << 22), slice(N - (1 << 22), N)):
        assert torch.equal(y[:, cols], part(a, w, slice(None), cols).bfloat16())
    assert not any(y[:, c:c + (1 << 27)].isnan().any() for c in range(0, N, 1 << 27))


@pytest.mark.parametrize("per, N", [(1, 60000), (2, 120000)])
def test_products_of_very_many_columns_of_groups(per, N):
    E = 4096
    a, w = random_rows(per * E, 16), random_rows(N, 16, E)
    y = torch.full((per * E, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    s3r.s3r_int_product(a, w, y, offsets=torch.arange(E + 1, device=DEV) * per)
    for e in (0, 1, 2047, 4094, 4095):
        rows = slice(per * e, per * e + per)
        assert torch.equal(y[rows], part(a, w, rows, slice(None), e).bfloat16())
    assert not any(y[r:r + 512].isnan().any() for r in range(0, per * E, 512))


@pytest.mark.parametrize("groups", [0, 2])
def test_products_of_the_most_rows(groups):
    M = (1 << 31) - 1
    a, w = random_rows(M, 5), random_rows(3, 5, max(groups, 1))
    a.codes[..., 5:] = 0
    offsets = torch.tensor([0, 7, M], device=DEV) if groups else None
    y = torch.full((M, 3), float("nan"), dtype=torch.bfloat16, device=DEV)
    s3r.s3r_int_product(a, w, y, offsets=offsets)
    e = 1 if groups else 0
    for rows in (slice(7, 1 << 20), slice(M // 2, M // 2 + (1 << 20)), slice(M - (1 << 20), M)):
        assert torch.equal(y[rows], part(a, w, rows, slice(None), e).bfloat16())
    assert torch.equal(y[:7], part(a, w, slice(0, 7), slice(None)).bfloat16())
    assert not any(y[r:r + (1 << 26)].isnan().any() for r in range(0, M, 1 << 26))


@pytest.mark.parametrize("M, N, K", [(1, 40, 2000), (4, 70, 300), (40, 60, 1100), (300, 270, 500)])
def test_rows_far_apart(M, N, K):
    """The largest leading dimensions (through the C ABI): codes of 2 GiB a tile."""
    ld = (1 << 23) - 16
    far_a, far_w = (torch.full((r, ld), 55, dtype=torch.int8, device=DEV) for r in (M, N))
    x, W = matrix((M, K), torch.float32, 1), matrix((N, K), torch.bfloat16, 2)
    w = s3r.int_rows(W)
    far_w[:, :K] = w.codes[0, :, :K]
    sa, y = torch.empty(M, device=DEV), torch.full((M, N), float("nan"), device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    L = s3r.lib()
    assert L.s3r_int_rows(1, M, K, x.data_ptr(), None, s3r.S3R_F32, K, 0, M, None, 1, far_a.data_ptr(), ld, 0, sa.data_ptr(),
                          None, stream) == 0
    d = s3r.IntPDesc(M, N, K, 0, ld, N * ld, s3r.S3R_F32, 0)
    assert L.s3r_int_product(d, far_a.data_ptr(), ld, sa.data_ptr(), None, far_w.data_ptr(), w.delta.data_ptr(), None,
                             y.data_ptr(), N, None, stream) == 0
    same(y, expected(x, w))
    pad = (K + 15) // 16 * 16
    assert not far_a[:, K:pad].any() and (far_a[:, pad:] == 55).all()
