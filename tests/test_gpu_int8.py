"""The W8A8 linear layer on the GPU: codes and scales bit-exact with the 64-bit
oracle, the product within its counted roundings, at the sizes where tiles,
slices of K and vector widths end."""
import ctypes

import numpy as np
import pytest
import torch

import block_oracle as B
from w4a4_diffusion_model_b200 import svdq as S

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    S.load()


def activations(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(K, generator=g))
    return (torch.randn(M, K, generator=g) * size).to(dtype)


def check_codes(x, mult, Q, s):
    q, sc = B.int8_codes(x.float().numpy(), None if mult is None else mult.numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), sc)
    np.testing.assert_array_equal(Q.cpu().numpy().astype(np.int64), q)


# one vector, rows of a warp, ragged warps, several vectors a thread, rows beyond the registers
@pytest.mark.parametrize("M,K", [(1, 16), (9, 48), (3, 512), (17, 1008), (5, 2064), (2, 4096), (3, 8208), (2, 16400),
                                 (2, 32784), (1, 131072), (4000, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_codes_are_exact(M, K, dtype):
    x = activations(M, K, dtype, M + K)
    mult = torch.exp(torch.randn(K, generator=torch.Generator().manual_seed(K)))
    for m in (None, mult):
        Q, s = S.svdq_int8_quantize_act(x.cuda(), None if m is None else m.cuda())
        check_codes(x, m, Q, s)


def test_codes_on_and_next_to_midpoints():
    """Scale 1 (maximum 127): every half-integer and its fp32 neighbours, both signs; and odd scales."""
    half = np.arange(0, 127, dtype=np.float32) + np.float32(0.5)
    near = [half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(1e3))]
    v = np.concatenate(near + [-n for n in near] + [np.arange(-127, 128, dtype=np.float32)])
    v = np.concatenate([v, np.zeros(-len(v) % 16, np.float32)])
    rows = [v, v * np.float32(2.0 ** -20)]
    for s in (np.float32(1.00001), np.float32(0.0123), np.float32(777.7)):     # products next to a midpoint of s
        rows.append(np.clip((v.astype(np.float64) * float(s)).astype(np.float32), -127 * s, 127 * s))
    x = torch.from_numpy(np.stack(rows))
    Q, s = S.svdq_int8_quantize_act(x.cuda())
    check_codes(x, None, Q, s)


def test_rows_of_zeros_tiny_values_and_what_is_not_finite():
    x = torch.randn(9, 64, generator=torch.Generator().manual_seed(5))
    x[0] = 0
    x[1] *= 1e-36
    x[2] = 0
    x[2, 3] = 1e-45                    # its scale rounds to 0
    x[3] *= 1e-42                      # a scale with few bits
    x[4] *= 1e37
    x[5, 7] = float("inf")
    x[6, 0] = float("nan")
    x[7, 63] = -float("inf")
    Q, s = S.svdq_int8_quantize_act(x.cuda())
    fine = [0, 1, 2, 3, 4, 8]
    check_codes(x[fine], None, Q[fine], s[fine])
    assert torch.isnan(s[5:8]).all() and not Q[5:8].any()
    W = S.svdq_int8_prepare_weights(torch.randn(24, 64).cuda())
    Y = S.svdq_int8_linear(Q, s, W, torch.float32)
    assert torch.isnan(Y[5:8]).all() and torch.isfinite(Y[fine]).all()


def check_product(M, K, N, dtype, bias, seed=0, stride=None):
    g = torch.Generator().manual_seed(seed + M * 7 + K * 3 + N)
    qx = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    qw = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g) * 0.02 + 1e-4, torch.rand(N, generator=g) * 0.002 + 1e-5
    b = torch.randn(N, generator=g) if bias else None
    W = S.Int8Weights(N, K, qw.cuda(), sw.cuda(), None, None if b is None else b.cuda())
    out = None
    if stride:   # columns of a wider matrix; the rest stays as it was
        wide = torch.full((M, stride), 7.0, dtype=dtype, device="cuda")
        out = wide[:, :N]
    Y = S.svdq_int8_linear(qx.cuda(), sx.cuda(), W, dtype, out=out)
    S.svdq_check()
    want, bound = B.int8_linear(qx.numpy(), sx.numpy(), qw.numpy(), sw.numpy(), None if b is None else b.numpy())
    B.within(Y, want, bound + B.rounding(want, dtype), f"Y {M}x{K}x{N}")
    if stride:
        assert (wide[:, N:] == 7).all()


# single rows and columns, K of one MMA step and below, a K tail, tiles that end inside, several tiles, N odd
SHAPES = [(1, 16, 1), (1, 128, 128), (2, 4096, 257), (7, 48, 33), (8, 144, 128), (77, 1360, 385), (127, 272, 129),
          (128, 256, 256), (129, 4112, 130), (256, 512, 512), (300, 640, 770), (513, 1024, 1032), (1, 13824, 5120),
          (1100, 160, 2051)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_product(M, K, N, dtype):
    check_product(M, K, N, dtype, bias=(M + N) % 2 == 0)


# each kernel and K split, as their sizes choose them: dot products for 1, 2, 4 and 8 tokens; a single CTA's tile with K
# whole, in halves, quarters and eighths; pairs whole and in halves; each with whole and ragged rows, columns and K
@pytest.mark.parametrize("M,K,N", [(1, 1040, 520), (2, 528, 1001), (3, 2064, 300), (7, 4112, 1030),
                                   (16, 4096, 24600), (40, 1360, 24577), (16, 4096, 12288), (13, 4112, 12289),
                                   (100, 4096, 5000), (77, 4240, 5003), (100, 4096, 1024), (33, 4112, 999), (1024, 1024, 2048), (700, 1104, 4097),
                                   (1024, 8192, 1024), (1100, 8208, 1033)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_route(M, K, N, dtype):
    check_product(M, K, N, dtype, bias=True, seed=5)


@pytest.mark.parametrize("M,K,N", [(5, 64, 40), (300, 256, 512), (130, 320, 136)])
@pytest.mark.parametrize("extra", [1, 4, 8])
def test_product_into_wider_rows(M, K, N, extra):
    for dtype in TYPES:
        check_product(M, K, N, dtype, True, stride=N + extra)


def test_unsmoothed_rows_whose_quotients_are_midpoints():
    """16-bit rows over maxima with short significands: 127 x / max is half an integer for many x."""
    g = torch.Generator().manual_seed(2)
    for dtype in TYPES[:2]:
        x = torch.randn(64, 1024, generator=g)
        top = torch.tensor([4.0, 3.9375, 3.96875, 3.0, 2.5, 127.0, 63.5, 254.0]).repeat(8)
        x = torch.minimum(torch.maximum(x, -top[:, None]), top[:, None])
        x[:, 0] = top
        x[32:, 1:] *= (top[32:] / 4)[:, None]
        x = x.to(dtype)
        Q, s = S.svdq_int8_quantize_act(x.cuda())
        check_codes(x, None, Q, s)


def test_many_rows_take_the_ring():
    """More rows than two per SM: rows streamed through shared memory, whole and ragged widths, strided."""
    for K in (528, 1024, 2064, 4096, 5136, 8192, 13824, 16384):
        M = 700 if K <= 4096 else 400
        x = activations(M, K + 16, torch.bfloat16, K)
        mult = torch.exp(torch.randn(K, generator=torch.Generator().manual_seed(K)))
        Q, s = S.svdq_int8_quantize_act(x.cuda()[:, 16:], mult.cuda())
        check_codes(x[:, 16:], mult, Q, s)
    x = activations(500, 1040, torch.float32, 9)
    Q, s = S.svdq_int8_quantize_act(x.cuda())
    check_codes(x, None, Q, s)


def test_extreme_codes_sum_exactly():
    """127 * 127 * 131072 < 2^31: the largest sums, of both signs, and codes of -128."""
    K = 131072
    qx = torch.full((2, K), 127, dtype=torch.int8)
    qx[1] = -127
    qw = torch.full((3, K), 127, dtype=torch.int8)
    qw[1] = -127
    qw[2] = -128
    W = S.Int8Weights(3, K, qw.cuda(), torch.ones(3).cuda())
    Y = S.svdq_int8_linear(qx.cuda(), torch.ones(2).cuda(), W, torch.float32)
    want = qx.numpy().astype(np.float64) @ qw.numpy().astype(np.float64).T
    np.testing.assert_array_equal(B.np64(Y), want.astype(np.float32).astype(np.float64))


def test_no_rows():
    W = S.svdq_int8_prepare_weights(torch.randn(8, 32).cuda())
    Q, s = S.svdq_int8_quantize_act(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"))
    assert S.svdq_int8_linear(Q, s, W).shape == (0, 8)


def test_smoothed_layer_end_to_end():
    """W8A8 of a layer prepared with the library's smoothing factors, rows of X inside a wider activation."""
    M, K, N = 200, 512, 384
    x = activations(M, K + 64, torch.bfloat16, 3)
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(4)) / K ** 0.5).to(torch.bfloat16)
    X = x.cuda()[:, 64:]
    P = S.svdq_prepare_weights(w.cuda(), S.svdq_channel_amax(X.contiguous()), 0.5, 0)
    W8 = S.svdq_int8_prepare_weights(w.cuda(), P.lam, P.inv_lam, torch.randn(N).to(torch.bfloat16).cuda())
    check_codes(w, P.lam.cpu(), W8.Qw, W8.Sw)
    Q, s = S.svdq_int8_quantize_act(X, W8.inv_lam)
    check_codes(x[:, 64:], P.inv_lam.cpu(), Q, s)
    Y = S.svdq_int8_linear(Q, s, W8)
    want, bound = B.int8_linear(Q.cpu().numpy(), s.cpu().numpy(), W8.Qw.cpu().numpy(), W8.Sw.cpu().numpy(),
                                W8.bias.cpu().numpy())
    B.within(Y, want, bound + B.rounding(want, torch.bfloat16))
    full = B.np64(x[:, 64:]) @ B.np64(w).T + B.np64(W8.bias)
    assert np.linalg.norm(B.np64(Y) - full) / np.linalg.norm(full) < 0.02     # 8 bits of the smoothed layer


@pytest.mark.parametrize("M,K,N", [(3, 256, 200), (300, 384, 520), (700, 512, 768)])
def test_guards_around_every_output(M, K, N):
    def guarded(n, dtype, shape):
        size = n * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((4096 + size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[4096:4096 + size].view(dtype).view(shape)
    x = activations(M, K, torch.bfloat16, 1).cuda()
    qb, Q = guarded(M * K, torch.int8, (M, K))
    sb, s = guarded(M, torch.float32, (M,))
    yb, Y = guarded(M * N, torch.bfloat16, (M, N))
    W = S.svdq_int8_prepare_weights(torch.randn(N, K).cuda())
    S.svdq_int8_quantize_act(x, out=(Q, s))
    S.svdq_int8_linear(Q, s, W, out=Y)
    S.svdq_check()
    for b in (qb, sb, yb):
        assert (b[:4096] == 0xA5).all() and (b[-4096:] == 0xA5).all()


def test_weights_quantized_on_the_stream_just_before():
    """The product follows the weights' quantizer on the stream with nothing in between, many times."""
    g = torch.Generator().manual_seed(12)
    for M, K, N in ((1, 1024, 512), (4, 4096, 2048), (32, 2048, 2048), (300, 512, 1024)):
        q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8).cuda()
        sx = torch.ones(M).cuda()
        ws = [torch.randn(N, K, generator=g).cuda() for _ in range(3)]
        prepared = [S.svdq_int8_prepare_weights(w) for w in ws]
        torch.cuda.synchronize()
        want = [S.svdq_int8_linear(q, sx, P) for P in prepared]
        torch.cuda.synchronize()
        W = prepared[0]
        for _ in range(4):
            for w, y in zip(ws, want):
                lib = S.load()
                st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
                assert lib.svdq_int8_quantize_weight(N, K, 2, w.data_ptr(), K, None, W.Qw.data_ptr(), W.Sw.data_ptr(), st) == 0
                assert torch.equal(S.svdq_int8_linear(q, sx, W), y)


def test_replayed_graph_and_other_stream():
    """A captured pair of calls replayed on new inputs, while another stream runs the same layer."""
    M, K, N = 64, 1024, 640
    W = S.svdq_int8_prepare_weights(torch.randn(N, K).cuda())
    X = activations(M, K, torch.bfloat16, 8).cuda()
    S.svdq_int8_linear(*S.svdq_int8_quantize_act(X), W)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = S.svdq_int8_linear(*S.svdq_int8_quantize_act(X), W)
    side = torch.cuda.Stream()
    for seed in (9, 10):
        X.copy_(activations(M, K, torch.bfloat16, seed))
        other = activations(M, K, torch.bfloat16, seed + 50).cuda()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            Z = S.svdq_int8_linear(*S.svdq_int8_quantize_act(other), W)
        torch.cuda.synchronize()
        assert torch.equal(Y, S.svdq_int8_linear(*S.svdq_int8_quantize_act(X), W))
        assert torch.equal(Z, S.svdq_int8_linear(*S.svdq_int8_quantize_act(other), W))


@pytest.mark.parametrize("M,N", [(2, 3), (40, 24), (600, 520)])
def test_codes_of_minus_128_on_both_sides(M, N):
    """128 * 128 * 131056 < 2^31, for each kind of kernel; at K = 131072 one side only."""
    for K, x in ((131056, -128), (131072, -127)):
        qx = torch.full((M, K), x, dtype=torch.int8, device="cuda")
        qx[1] = 127
        qw = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        W = S.Int8Weights(N, K, qw, torch.ones(N, device="cuda"))
        Y = S.svdq_int8_linear(qx, torch.ones(M, device="cuda"), W, torch.float32)
        want = torch.full((M, N), -128.0 * x * K, dtype=torch.float64)
        want[1] = -128.0 * 127 * K
        assert torch.equal(Y.cpu(), want.float())


@pytest.mark.parametrize("dtype", TYPES)
def test_scales_and_codes_next_to_the_exact_quotients(dtype):
    """max / 127 in 64 bits: fp32(1/127) is (1/127) (1 - 2^-28), so that the scale is off by half a step and a sixteenth at
    most, and a code by what that makes of 127 v / max; and the same scales from torch's own division on the GPU."""
    x = activations(3000, 64, dtype, 21)
    x *= torch.exp(torch.randn(3000, 1, generator=torch.Generator().manual_seed(22))).to(dtype)
    x[:2] = 0
    x[0, 5] = 127.0
    x[1, 5] = torch.finfo(dtype).tiny
    X = x.cuda()
    Q, s = S.svdq_int8_quantize_act(X)
    v, sc = B.np64(x), B.np64(s)
    top = np.abs(v).max(1)
    assert (np.abs(sc - top / 127) <= (0.5 + 1 / 16) * np.spacing(s.cpu().numpy()).astype(np.float64)).all()
    rounded = (top / 127).astype(np.float32)
    differ = s.cpu().numpy() != rounded
    assert (np.abs(sc - rounded)[differ] <= np.spacing(rounded[differ])).all()
    normal = top / 127 >= np.finfo(np.float32).tiny          # below, a step is more than 2^-23 of the scale
    off = 127 * (2.0 ** -24 + 2.0 ** -28) * (1 + 2.0 ** -20)
    assert (np.abs(B.np64(Q.double()) - 127 * v / top[:, None])[normal] <= 0.5 + off).all()
    assert torch.equal(s, X.float().abs().amax(1) / 127.0)


# rows of Y that end inside a 16-byte piece of a wider matrix whose rows begin on one: pairs whole and in halves of K
@pytest.mark.parametrize("M,K,N", [(399, 128, 95), (241, 16, 3), (1265, 32, 4), (300, 256, 100), (1100, 8208, 1033),
                                   (40, 512, 30), (7, 256, 22)])
@pytest.mark.parametrize("dtype", TYPES)
def test_product_leaves_what_is_behind_its_columns(M, K, N, dtype):
    piece = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = N + (-N % piece or piece)
    check_product(M, K, N, dtype, True, stride=ld)
    # the last row ends with the memory that belongs to Y
    size = (M - 1) * ld + N
    buf = torch.full((size + 4 * piece,), 7.0, dtype=dtype, device="cuda")
    Y = buf.as_strided((M, N), (ld, 1))
    W = S.Int8Weights(N, K, torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"))
    S.svdq_int8_linear(torch.ones(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"), W, out=Y)
    assert (Y == torch.tensor(K, dtype=dtype)).all() and (buf[size:] == 7).all()
