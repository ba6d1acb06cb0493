"""Layer norm on the GPU: forward, backward and the form that ends in 8-bit
codes, against the 64-bit oracle within counted roundings."""
import numpy as np
import pytest
import torch

import block_oracle as B
from w4a4_diffusion_model_b200 import svdq as S

pytestmark = pytest.mark.gpu
BF, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    S.load()


def case(M, C, dtype, wtype, groups, seed=0, rows=None):
    g = torch.Generator().manual_seed(seed + 31 * M + C)
    x = torch.randn(M, C, generator=g) * torch.exp(0.5 * torch.randn(C, generator=g)) + 0.5 * torch.randn(C, generator=g)
    shape = (C,) if groups is None else (groups, C)
    w = torch.randn(shape, generator=g) * 0.5 + 0.5
    b = torch.randn(shape, generator=g)
    dy = torch.randn(M, C, generator=g)
    return x.to(dtype), w.to(wtype), b.to(wtype), dy.to(dtype)


def run(x, w, b, dy, rows=None, add_one=False, eps=1e-6):
    dtype = x.dtype
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    X, W, Bb, dY = c(x), c(w), c(b), c(dy)
    Y, mean, rstd = S.svdq_layernorm(X, W, Bb, eps, rows, add_one)
    M, C = x.shape
    n = 0 if w is None or w.dim() == 1 else rows or M // w.shape[0]
    n64 = lambda t: None if t is None else B.np64(t)  # noqa: E731
    y, mu, r, by, bmu, br = B.layernorm(B.np64(x), n64(w), n64(b), eps, n, add_one)
    B.within(mean, mu, bmu + B.U * np.abs(mu) + 2.0 ** -140, "mean")
    B.within(rstd, r, br + B.U * r, "rstd")
    B.within(Y, y, by + B.rounding(y, dtype), "Y")
    dX, dw, db = S.svdq_layernorm_backward(dY, X, W, mean, rstd, rows, add_one)
    dx, gw, gb, bx, bw, bb = B.layernorm_backward(B.np64(dy), B.np64(x), n64(w), B.np64(mean), B.np64(rstd), n, add_one)
    B.within(dX, dx, bx + B.rounding(dx, dtype), "dX")
    shape = (C,) if w is None else w.shape
    assert dw.shape == shape and db.shape == shape
    B.within(dw, gw.reshape(shape), bw.reshape(shape) + B.rounding(gw.reshape(shape), FP32), "dweight")
    B.within(db, gb.reshape(shape), bb.reshape(shape) + B.rounding(gb.reshape(shape), FP32), "dbias")
    return Y, mean, rstd, dX, dw, db


# widths of one value, below and above a warp, ragged, of several vectors, the largest; rows from one up
@pytest.mark.parametrize("M,C", [(1, 1), (5, 3), (3, 8), (33, 64), (2, 255), (10, 1152), (37, 1151), (4, 2048),
                                 (19, 2050), (6, 4096), (3, 5120), (2, 8192), (2, 16384), (2, 16383), (700, 96),
                                 (1301, 40)])
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (BF, FP32), (FP16, FP16), (FP16, FP32), (FP32, FP32)])
def test_affine(M, C, dtype, wtype):
    run(*case(M, C, dtype, wtype, None))


@pytest.mark.parametrize("M,C,groups,rows", [(8, 64, 2, None), (600, 256, 3, None), (7, 48, 7, None),
                                             (10, 32, 3, 4), (9, 33, 2, 8), (2000, 128, 2, None), (300, 16, 300, None)])
@pytest.mark.parametrize("add_one", [False, True])
def test_modulated_groups(M, C, groups, rows, add_one):
    for dtype, wtype in ((BF, BF), (FP32, FP32), (FP16, FP32)):
        run(*case(M, C, dtype, wtype, groups), rows=rows, add_one=add_one)


def test_without_weight_or_bias():
    x, w, b, dy = case(12, 136, BF, BF, None)
    run(x, None, None, dy)
    run(x, w, None, dy)
    Y, *_ = S.svdq_layernorm(x.cuda(), None, b.cuda())
    y, *_, = B.layernorm(B.np64(x), None, B.np64(b), 1e-6, 0, False)
    by = B.layernorm(B.np64(x), None, B.np64(b), 1e-6, 0, False)[3]
    B.within(Y, y, by + B.rounding(y, BF))


def test_rows_with_large_means_and_constant_rows():
    """The variance is taken around the mean: a mean of 1000 deviations costs no more than its bound, a constant row
    has variance 0 and a finite gradient."""
    x, w, b, dy = case(6, 512, FP32, FP32, None)
    x[0] += 1000
    x[1] = 3.0
    x[2] = 0.0
    Y, mean, rstd, dX, *_ = run(x, w, b, dy, eps=1e-5)
    assert torch.equal(Y[1:3].cpu(), b.expand(2, -1)) and torch.isfinite(dX).all()


def test_nan_and_infinity_stay_in_their_rows():
    x, w, b, dy = case(5, 200, FP32, FP32, None)
    clean = S.svdq_layernorm(x.cuda(), w.cuda(), b.cuda())[0]
    x[1, 3], x[3, 199] = float("nan"), float("inf")
    Y = S.svdq_layernorm(x.cuda(), w.cuda(), b.cuda())[0]
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[3]).any()
    assert torch.equal(Y[[0, 2, 4]], clean[[0, 2, 4]])


@pytest.mark.parametrize("C,pad", [(64, 8), (64, 3), (1152, 16), (130, 1)])
def test_strided_rows_and_in_place(C, pad):
    x, w, b, dy = case(21, C, BF, BF, None)
    Y, mean, rstd = S.svdq_layernorm(x.cuda(), w.cuda(), b.cuda())
    dX, dw, db = S.svdq_layernorm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    wide = torch.full((21, C + pad), 5.0, dtype=BF, device="cuda")
    X = wide[:, :C]
    X.copy_(x)
    assert torch.equal(S.svdq_layernorm(X, w.cuda(), b.cuda())[0], Y)
    grad = torch.full((21, C + pad), 5.0, dtype=BF, device="cuda")
    G = grad[:, :C]
    G.copy_(dy)
    got = S.svdq_layernorm_backward(G, X, w.cuda(), mean, rstd, out=G)
    assert torch.equal(G, dX) and torch.allclose(got[1], dw, rtol=1e-5, atol=1e-5)
    S.svdq_layernorm(X, w.cuda(), b.cuda(), out=X)
    assert torch.equal(X, Y) and (wide[:, C:] == 5).all() and (grad[:, C:] == 5).all()


# more rows than two per SM: rows streamed through the ring, in each of its widths, whole and ragged
@pytest.mark.parametrize("C", [520, 1024, 2048, 2056, 4096, 4104, 5120, 8192, 12288, 16384])
def test_many_rows(C):
    M = 600 if C <= 5120 else 310
    for dtype, wtype, groups in ((BF, BF, 2), (FP32, FP32, None)):
        run(*case(M, C, dtype, wtype, groups), add_one=groups is not None)


@pytest.mark.parametrize("C", [515, 2047, 2051, 2060, 4099, 9001])
def test_many_rows_of_odd_widths(C):
    run(*case(320, C, BF, FP32, 2), add_one=True)
    run(*case(303, C, FP32, FP32, None))


def test_many_groups_of_many_rows():
    run(*case(1200, 1024, BF, FP32, 240))
    run(*case(1203, 640, FP16, FP16, 241), rows=5)


@pytest.mark.parametrize("M,C", [(40, 96), (700, 96), (200, 1160), (700, 1160), (340, 9000), (300, 2057), (300, 2060)])
def test_gradient_in_the_memory_of_either_input(M, C):
    x, w, b, dy = (t.cuda() for t in case(M, C, BF, BF, None))
    _, mean, rstd = S.svdq_layernorm(x, w, b)
    want = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    for which in (0, 1):
        a = [dy.clone(), x.clone()]
        got = S.svdq_layernorm_backward(a[0], a[1], w, mean, rstd, out=a[which])
        for p, q in zip(want, got):
            assert torch.equal(p, q)


def test_only_the_gradient_of_the_input():
    for M in (40, 800):
        x, w, b, dy = (t.cuda() for t in case(M, 200, BF, BF, None))
        _, mean, rstd = S.svdq_layernorm(x, w, b)
        want = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
        dX, dw, db = S.svdq_layernorm_backward(dy, x, w, mean, rstd, params=False)
        assert torch.equal(dX, want[0]) and dw is None and db is None


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    Y, mean, rstd = S.svdq_layernorm(x, w)
    dX, dw, db = S.svdq_layernorm_backward(Y, x, w, mean, rstd)
    assert Y.shape == dX.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (64,)


def test_two_calls_give_the_same_bits():
    x, w, b, dy = (t.cuda() for t in case(3000, 384, BF, FP32, 3))
    _, mean, rstd = S.svdq_layernorm(x, w, b)
    first = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        for a, c in zip(first, S.svdq_layernorm_backward(dy, x, w, mean, rstd)):
            assert torch.equal(a, c)


def test_gradient_against_differences():
    """dX, dweight and dbias of sum(Y * dY) against central differences of the forward pass in fp64."""
    x, w, b, dy = case(4, 24, FP32, FP32, 2)
    eps = 1e-6
    _, mean, rstd = S.svdq_layernorm(x.cuda(), w.cuda(), b.cuda(), eps, add_one=True)
    dX, dw, db = S.svdq_layernorm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, add_one=True)

    def loss(xx, ww, bb):
        return (B.layernorm(xx, ww, bb, eps, 2, True)[0] * B.np64(dy)).sum()

    args = [B.np64(x), B.np64(w), B.np64(b)]
    step = 1e-5
    for k, got in enumerate((dX, dw, db)):
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][i] += step
            lo[k][i] -= step
            num[i] = (loss(*hi) - loss(*lo)) / (2 * step)
        # truncation step^2 f''' / 6 and cancellation 2^-52 |loss| / step, both far below 1e-5; fp32 adds its steps
        np.testing.assert_allclose(B.np64(got), num, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("M,C", [(1, 16), (9, 1152), (300, 2048), (400, 1168), (5, 5120), (3, 16384), (310, 8208)])
@pytest.mark.parametrize("dtype", [BF, FP16, FP32])
def test_norm_into_codes(M, C, dtype):
    """Scales within the norm's roundings; a code off by one only where the exact quotient is that near a midpoint."""
    x, w, b, _ = case(M, C, dtype, dtype, 1)
    lam = torch.exp(0.3 * torch.randn(C, generator=torch.Generator().manual_seed(C)))
    Q, s = S.svdq_int8_layernorm_quantize(x.cuda(), w.cuda(), b.cuda(), lam.cuda(), add_one=True)
    y, *_, = B.layernorm(B.np64(x), B.np64(w), B.np64(b), 1e-6, 0, True)
    by = B.layernorm(B.np64(x), B.np64(w), B.np64(b), 1e-6, 0, True)[3]
    v, bv = y * B.np64(lam), by * B.np64(lam) + B.U * np.abs(y * B.np64(lam))
    top = np.abs(v).max(1)
    B.within(s, top / 127, bv.max(1) / 127 + 2 * B.U * top / 127, "scale")
    sg = B.np64(s)[:, None]
    # |code - v / s| is half a step, and what v and the quotient's own settling may be off
    B.within(Q.double(), v / sg, 0.5 + bv / sg + 1e-9, "codes")


@pytest.mark.parametrize("M,C", [(50, 768), (700, 768), (700, 4096)])
def test_norm_into_codes_matches_the_two_calls_in_fp32(M, C):
    x, w, b, _ = case(M, C, FP32, FP32, None)
    Y, *_ = S.svdq_layernorm(x.cuda(), w.cuda(), b.cuda())
    Q2, s2 = S.svdq_int8_quantize_act(Y)
    Q, s = S.svdq_int8_layernorm_quantize(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(Q, Q2) and torch.equal(s, s2)      # fp32 Y has nothing to lose


def test_captured_backward():
    x, w, b, dy = (t.cuda() for t in case(500, 256, BF, BF, 2))
    _, mean, rstd = S.svdq_layernorm(x, w, b)
    S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, mean, rstd = S.svdq_layernorm(x, w, b)
        out = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    x.mul_(1.5)
    dy.add_(0.25)
    graph.replay()
    _, m2, r2 = S.svdq_layernorm(x, w, b)
    for a, c in zip(out, S.svdq_layernorm_backward(dy, x, w, m2, r2)):
        assert torch.equal(a, c)


# off 16-byte boundaries, many rows: one warp a row (4 and 8 values a thread), several rows of several warps in a
# block, one row, sixteen warps; rows that leave teams and chunks idle
@pytest.mark.parametrize("M,C", [(701, 1), (1203, 51), (997, 127), (1501, 129), (1400, 251), (650, 571), (1100, 1151),
                                 (420, 2044), (403, 2049), (450, 4090), (405, 4095)])
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (FP16, FP32), (FP32, FP32)])
def test_single_values(M, C, dtype, wtype):
    if C % (4 if dtype == FP32 else 8) == 0:
        pytest.skip("fits 16-byte pieces")
    run(*case(M, C, dtype, wtype, None, 1))


@pytest.mark.parametrize("M,C,groups,rows", [(903, 51, 3, None), (1404, 381, 4, None), (1000, 381, 3, 401),
                                             (405, 571, 405, None), (502, 1151, 2, None), (460, 2501, 230, None)])
@pytest.mark.parametrize("add_one", [False, True])
def test_single_values_in_groups(M, C, groups, rows, add_one):
    run(*case(M, C, BF, FP32, groups, 2), rows=rows, add_one=add_one)


@pytest.mark.parametrize("M,C,pad", [(900, 120, 3), (700, 571, 0), (500, 3000, 1)])
def test_single_values_in_place(M, C, pad):
    """Strides off 16-byte boundaries; the next row is loaded before this one's result is stored over it."""
    x, w, b, dy = case(M, C, BF, BF, None, 3)
    _, mean, rstd, *_ = run(x, w, b, dy)
    X, dY = (torch.empty(M, C + pad, dtype=BF, device="cuda")[:, :C].copy_(t) for t in (x, dy))
    W = w.cuda()
    got, gw, gb = S.svdq_layernorm_backward(dY, X, W, mean, rstd)
    over, ow, ob = S.svdq_layernorm_backward(dY, X, W, mean, rstd, out=dY)
    assert over.data_ptr() == dY.data_ptr() and torch.equal(over, got) and torch.equal(ow, gw) and torch.equal(ob, gb)
    out, m2, r2 = S.svdq_layernorm(X, W, b.cuda())
    same, m3, r3 = S.svdq_layernorm(X, W, b.cuda(), out=X)
    assert same.data_ptr() == X.data_ptr() and torch.equal(same, out) and torch.equal(m2, m3) and torch.equal(r2, r3)


@pytest.mark.parametrize("C", [51, 381, 1151, 2501])
def test_single_values_with_large_means(C):
    """The variance of values far from zero, and of a column range that differs from the rest."""
    x, w, b, dy = case(450, C, FP32, FP32, None, 4)
    x[::2] += 1000.0
    x[1::2, : C // 3] += 500.0
    run(x, w, b, dy)


@pytest.mark.parametrize("C", [381, 1151, 2501])
def test_single_values_nan_and_infinity_stay_in_their_rows(C):
    x, w, b, dy = (t.cuda() for t in case(600, C, BF, BF, None, 5))
    Y, mean, rstd = S.svdq_layernorm(x, w, b)
    dX, *_ = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    z = x.clone()
    z[7, 3], z[500, C - 1] = float("nan"), float("inf")
    Y2, mean2, rstd2 = S.svdq_layernorm(z, w, b)
    dX2, *_ = S.svdq_layernorm_backward(dy, z, w, mean2, rstd2)
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[[7, 500]] = False
    assert torch.equal(Y[keep], Y2[keep]) and torch.equal(dX[keep], dX2[keep])
    assert Y2[~keep].isnan().all() and dX2[~keep].isnan().all()


# 16-bit rows of four-value pieces, wider than the forms for single values take, and rows that a stride puts off 16-byte
# boundaries, at row counts that leave the few-rows limits
@pytest.mark.parametrize("M,C,dtype", [(700, 5124, BF), (600, 9004, FP16), (410, 16380, BF), (700, 5124, FP32)])
def test_wide_rows_of_half_pieces(M, C, dtype):
    run(*case(M, C, dtype, FP32, 2, 6), add_one=True)


@pytest.mark.parametrize("M,C,pad,groups", [(500, 64, 0, 1), (700, 381, 0, 2), (700, 1152, 0, 1), (700, 1152, 3, 1),
                                            (450, 4096, 0, 2), (450, 4096, 1, 2), (420, 5124, 0, 1), (420, 8192, 5, 1)])
@pytest.mark.parametrize("dtype", [BF, FP32])
def test_nothing_is_written_past_the_workspace(M, C, pad, groups, dtype):
    x, w, b, dy = (t.cuda() for t in case(M, C, dtype, FP32, groups, 7))
    _, mean, rstd = S.svdq_layernorm(x, w, b)
    want = S.svdq_layernorm_backward(dy, x, w, mean, rstd)
    X, dY, dX = (torch.empty(M, C + pad, dtype=dtype, device="cuda")[:, :C].copy_(t) for t in (x, dy, x))
    dw, db = torch.empty_like(w), torch.empty_like(w)
    need = S.svdq_layernorm_backward_workspace(M, C, M // groups)
    work = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    t = S.DTYPES[dtype]
    status = S.load().svdq_layernorm_backward(M, C, t, S.DTYPES[FP32], dY.data_ptr(), C + pad, X.data_ptr(), C + pad,
                                              w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), M // groups, 0,
                                              dX.data_ptr(), C + pad, dw.data_ptr(), db.data_ptr(), work.data_ptr(), need,
                                              torch.cuda.current_stream().cuda_stream)
    assert status == 0 and (work[need:] == 0xA5).all()
    args = B.np64(dy), B.np64(x), B.np64(w), B.np64(mean), B.np64(rstd), M // groups, False
    dx, gw, gb, bx, bw, bb = B.layernorm_backward(*args)
    B.within(dX, dx, bx + B.rounding(dx, dtype), "dX")
    B.within(dw, gw, bw + B.rounding(gw, FP32), "dweight")
    B.within(db, gb, bb + B.rounding(gb, FP32), "dbias")
    assert torch.equal(want[0], dX) or pad


# every width of the forms for single values (strides off 16 bytes) and of whole pieces, one row a block and the ring
@pytest.mark.parametrize("C", [16, 1152, 4096, 8208, 16384])
@pytest.mark.parametrize("M,rows", [(7, 4), (400, 150)])
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (FP16, FP32), (FP32, FP32)])
def test_norm_into_codes_of_strided_rows_in_groups(C, M, rows, dtype, wtype):
    groups = -(-M // rows)
    x, w, b, _ = case(M, C, dtype, wtype, groups, 8)
    lam = torch.exp(0.3 * torch.randn(C, generator=torch.Generator().manual_seed(C + 1)))
    y, _, _, by, _, _ = B.layernorm(B.np64(x), B.np64(w), B.np64(b), 1e-6, rows, True)
    v, bv = y * B.np64(lam), by * B.np64(lam) + B.U * np.abs(y * B.np64(lam))
    top, dense = np.abs(v).max(1), None
    for pad in (0, 16, 3):
        X = torch.empty(M, C + pad, dtype=dtype, device="cuda")[:, :C].copy_(x)
        Q, s = S.svdq_int8_layernorm_quantize(X, w.cuda(), b.cuda(), lam.cuda(), rows_per_group=rows, add_one=True)
        if pad == 16:      # whole pieces all the same: the dense rows' order of sums
            assert torch.equal(Q, dense[0]) and torch.equal(s, dense[1])
        dense = dense or (Q, s)
        B.within(s, top / 127, bv.max(1) / 127 + 2 * B.U * top / 127, "scale")
        sg = B.np64(s)[:, None]
        B.within(Q.double(), v / sg, 0.5 + bv / sg + 1e-9, "codes")


def test_norm_of_streamed_rows_in_their_own_memory():
    """Rows that run through the ring, Y over X and strided: the rows ahead are on their way as a row is stored."""
    for C, pad in ((1024, 0), (4096, 8), (8200, 24)):
        x, w, b, _ = case(700, C, BF, BF, 2, 9)
        X = torch.full((700, C + pad), 3.0, dtype=BF, device="cuda")
        X[:, :C] = x.cuda()
        Y, mean, rstd = S.svdq_layernorm(X[:, :C], w.cuda(), b.cuda(), add_one=True)
        got = S.svdq_layernorm(X[:, :C], w.cuda(), b.cuda(), add_one=True, out=X[:, :C])
        assert torch.equal(X[:, :C], Y) and torch.equal(got[1], mean) and torch.equal(got[2], rstd)
        assert (X[:, C:] == 3).all()
