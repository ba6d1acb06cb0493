"""The operators around the 4-bit linear layer run together, as a transformer
block uses them: modulated norm into 8-bit codes, the merged QKV product, the
rotation of the query and key heads in place; and the way back through the
rotation and the norm. Each stage is checked on what the stage before it gave,
and the whole against the block in 64 bits within the quantizers' own steps."""
import numpy as np
import pytest
import torch

import block_oracle as B
from w4a4_diffusion_model_b200 import svdq as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    S.load()


class Block:
    """Two images of `side` x `side` tokens after `text` text tokens, heads of D with three axes."""

    def __init__(self, side, text, heads, D, dims, seed):
        g = torch.Generator().manual_seed(seed)
        self.C, self.heads, self.D, self.per = heads * D, heads, D, text + side * side
        M = 2 * self.per
        self.x = (torch.randn(M, self.C, generator=g) * torch.exp(0.5 * torch.randn(self.C, generator=g))).to(torch.bfloat16)
        self.scale = (0.3 * torch.randn(2, self.C, generator=g)).to(torch.bfloat16)
        self.shift = (0.3 * torch.randn(2, self.C, generator=g)).to(torch.bfloat16)
        self.w = (torch.randn(3 * self.C, self.C, generator=g) / self.C ** 0.5).to(torch.bfloat16)
        self.bias = torch.randn(3 * self.C, generator=g)
        t = torch.arange(side * side)
        grid = torch.stack([torch.zeros_like(t), t // side, t % side], 1)
        self.pos = torch.cat([torch.zeros(text, 3, dtype=torch.int64), grid]).to(torch.int32)
        self.table = S.svdq_rope_table(dims)
        self.X, self.sc, self.sh, self.P = self.x.cuda(), self.scale.cuda(), self.shift.cuda(), self.pos.cuda()
        amax = S.svdq_channel_amax(S.svdq_layernorm(self.X, self.sc, self.sh, add_one=True)[0])
        prepared = S.svdq_prepare_weights(self.w.cuda(), amax, 0.5, 0)
        self.lam = prepared.lam
        self.W8 = S.svdq_int8_prepare_weights(self.w.cuda(), prepared.lam, prepared.inv_lam, self.bias.cuda())

    def forward(self):
        Q, s = S.svdq_int8_layernorm_quantize(self.X, self.sc, self.sh, self.W8.inv_lam, add_one=True)
        Y = S.svdq_int8_linear(Q, s, self.W8)
        qkv = Y.view(-1, 3 * self.heads, self.D)
        qk = qkv[:, :2 * self.heads]
        S.svdq_rope(qk, self.P, self.table, out=qk)      # a batch shares its positions
        return Q, s, qkv


@pytest.mark.parametrize("side,text,heads,D,dims", [(4, 3, 4, 64, (16, 24, 24)), (16, 77, 6, 128, (16, 56, 56))])
def test_block_forward(side, text, heads, D, dims):
    blk = Block(side, text, heads, D, dims, seed=side)
    Q, s, qkv = blk.forward()
    S.svdq_check()
    y, _, _, by, _, _ = B.layernorm(B.np64(blk.x), B.np64(blk.scale), B.np64(blk.shift), 1e-6, blk.per, True)
    inv = B.np64(blk.W8.inv_lam)
    v, bv = y * inv, by * inv + B.U * np.abs(y * inv)
    sx = B.np64(s)[:, None]
    B.within(Q.double(), v / sx, 0.5 + bv / sx + 1e-9, "codes")
    Y = S.svdq_int8_linear(Q, s, blk.W8)
    want, bound = B.int8_linear(Q.cpu().numpy(), s.cpu().numpy(), blk.W8.Qw.cpu().numpy(), blk.W8.Sw.cpu().numpy(),
                                blk.bias.numpy())
    B.within(Y, want, bound + B.rounding(want, torch.bfloat16), "QKV")
    qk = B.np64(Y).reshape(len(Y), 3 * heads, D)[:, :2 * heads]
    turned, rb = B.rope(qk, B.np64(blk.pos), dims, B.np64(blk.table.freqs), True, False)
    B.within(qkv[:, :2 * heads], turned, rb + B.rounding(turned, torch.bfloat16), "rotated")
    assert torch.equal(qkv[:, 2 * heads:].reshape(len(Y), -1), Y[:, 2 * heads * D:])
    # the whole product against the block without quantization: half a step of each code is all that is lost
    lam, w = B.np64(blk.lam), B.np64(blk.w)
    what, sw = w * lam, B.np64(blk.W8.Sw)
    exact = v @ what.T + B.np64(blk.bias)
    kept = B.np64(blk.W8.Qw) * sw[:, None]
    slack = (0.5 * sx + bv) @ np.abs(kept).T + np.abs(v) @ (0.5 * (1 + 2.0 ** -20) * sw[:, None] + np.zeros_like(what)).T
    B.within(Y, exact, slack + 2 * bound + B.rounding(exact, torch.bfloat16) + B.HALF_STEP[torch.bfloat16] * slack, "block")


def test_block_backward():
    """<dOut, rope(norm(x))> back to x, scale and shift: the two gradients chained, against differences in 64 bits."""
    T, heads, D, dims = 10, 2, 16, (4, 6, 6)
    g = torch.Generator().manual_seed(7)
    C = heads * D
    x, dout = torch.randn(T, C, generator=g), torch.randn(T, C, generator=g)
    scale, shift = 0.3 * torch.randn(2, C, generator=g), torch.randn(2, C, generator=g)
    pos = torch.randint(0, 50, (T, 3), generator=g, dtype=torch.int32)
    table = S.svdq_rope_table(dims)
    X, W = x.cuda(), scale.cuda()
    _, mean, rstd = S.svdq_layernorm(X, W, shift.cuda(), add_one=True)
    dY = S.svdq_rope(dout.cuda().view(T, heads, D), pos.cuda(), table, inverse=True).view(T, C)
    grads = S.svdq_layernorm_backward(dY, X, W, mean, rstd, add_one=True)

    def loss(a):
        y = B.layernorm(a[0], a[1], a[2], 1e-6, 5, True)[0].reshape(T, heads, D)
        return (B.rope(y, B.np64(pos), dims, B.np64(table.freqs), True, False)[0].reshape(T, C) * B.np64(dout)).sum()

    args, step = [B.np64(x), B.np64(scale), B.np64(shift)], 1e-5
    for k, got in enumerate(grads):
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][i] += step
            lo[k][i] -= step
            num[i] = (loss(hi) - loss(lo)) / (2 * step)
        # differences: truncation step^2 f'''/6 and 2^-52 |loss| / step, far below 1e-5; fp32 adds its steps
        np.testing.assert_allclose(B.np64(got), num, rtol=1e-4, atol=1e-4)


def test_block_captured_and_on_other_streams():
    """The block in two graphs that replay at once on two streams, with inputs that change between replays."""
    blocks = [Block(6, 5, 4, 64, (16, 24, 24), seed=k) for k in (1, 2)]
    streams, graphs, outs = [torch.cuda.Stream() for _ in blocks], [], []
    for blk, st in zip(blocks, streams):
        blk.forward()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            outs.append(blk.forward())
        graphs.append(graph)
    for turn in range(3):
        for blk in blocks:
            blk.X.mul_(1.25)
            blk.sh.add_(0.125)
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for blk, out in zip(blocks, outs):
            for a, b in zip(out, blk.forward()):
                assert torch.equal(a, b), turn


def test_calls_ahead_of_the_4bit_layer():
    """The norm in front of the NVFP4 quantizer and GEMM: programmatic launches of both kinds follow one another."""
    g = torch.Generator().manual_seed(3)
    X = torch.randn(300, 512, generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn(256, 512, generator=g) / 22).to(torch.bfloat16).cuda()
    Y, *_ = S.svdq_layernorm(X)
    P = S.svdq_prepare_weights(W, S.svdq_channel_amax(Y), 0.5, 16)
    torch.cuda.synchronize()
    want = None
    for _ in range(5):
        Y, *_ = S.svdq_layernorm(X)
        Qx, Sx, T = S.svdq_quantize_act(Y, P.inv_lam, P.L1p, 16, 256)
        out = S.svdq_layernorm(S.svdq_linear(Qx, Sx, T, P))[0]
        S.svdq_check()
        if want is None:
            want = out
        assert torch.equal(out, want)


def test_tensors_of_one_call_live_on_one_device():
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError, match="one CUDA device"):
        S.svdq_layernorm(x, torch.ones(64))
    with pytest.raises(ValueError, match="contiguous"):
        S.svdq_layernorm(x, torch.ones(128, device="cuda")[::2])
    with pytest.raises(ValueError, match="rows"):
        S.svdq_layernorm(x.t())
    with pytest.raises(ValueError, match="groups"):
        S.svdq_layernorm(x, torch.ones(3, 64, device="cuda"))
    with pytest.raises(ValueError, match="out must"):
        S.svdq_layernorm(x, out=torch.empty(4, 32, device="cuda"))
    with pytest.raises(S.SvdqError, match="SHAPE"):
        S.svdq_int8_quantize_act(torch.randn(4, 40, device="cuda"))
    with pytest.raises(ValueError, match="bf16, fp16 or fp32"):
        S.svdq_int8_quantize_act(torch.zeros(4, 64, dtype=torch.int8, device="cuda"))
    with pytest.raises(S.SvdqError, match="overlap"):
        S.svdq_rope(torch.randn(4, 2, 16, device="cuda"), torch.zeros(4, 1, dtype=torch.int32, device="cuda"),
                    S.svdq_rope_table((16,)), out=torch.empty(4, 1, 16, device="cuda").expand(4, 2, 16))


def test_offsets_past_32_bits():
    """More than 2^31 elements in every matrix: the last rows give the bits that they give in a call of their own."""
    M, C, last, bf16 = 142_008, 15_360, 1000, torch.bfloat16
    assert (M - last) * C > 2 ** 31
    x = torch.empty(M, C, dtype=bf16, device="cuda").normal_()
    w, b = torch.randn(2, C, device="cuda"), torch.randn(2, C, device="cuda")
    half = M // 2
    tail = w[1].contiguous(), b[1].contiguous()
    Y, mean, rstd = S.svdq_layernorm(x, w, b)
    for a, c in zip((Y, mean, rstd), S.svdq_layernorm(x[-last:], *tail)):
        assert torch.equal(a[-last:], c)
    dX, _, db = S.svdq_layernorm_backward(Y, x, w, mean, rstd)
    dX2, *_ = S.svdq_layernorm_backward(Y[-last:], x[-last:], tail[0], mean[-last:].clone(), rstd[-last:].clone())
    assert torch.equal(dX[-last:], dX2)
    want = torch.stack([Y[k * half:(k + 1) * half].sum(0, dtype=torch.float64) for k in (0, 1)])
    size = torch.stack([Y[k * half:(k + 1) * half].float().abs().sum(0) for k in (0, 1)]).double()
    # a column's sum passes at most half / 4 + 24 additions in turn
    assert ((db.double() - want).abs() <= (half / 4 + 24) * B.U * size).all()
    del Y, dX
    Q, s = S.svdq_int8_layernorm_quantize(x, w, b)
    for a, c in zip((Q, s), S.svdq_int8_layernorm_quantize(x[-last:], *tail)):
        assert torch.equal(a[-last:], c)
    Q, s = S.svdq_int8_quantize_act(x)
    for a, c in zip((Q, s), S.svdq_int8_quantize_act(x[-last:])):
        assert torch.equal(a[-last:], c)
    del Q
    W = S.svdq_int8_prepare_weights(torch.randn(C, 64, device="cuda"))
    Q, s = S.svdq_int8_quantize_act(x[:, :64])
    S.svdq_int8_linear(Q, s, W, out=x)
    assert torch.equal(x[-last:], S.svdq_int8_linear(Q[-last:], s[-last:].clone(), W))
    table, pos = S.svdq_rope_table((16, 16)), torch.arange(M, dtype=torch.int32, device="cuda").view(-1, 1).repeat(1, 2)
    heads = x.view(M, -1, 64)
    want = S.svdq_rope(heads[-last:], pos[-last:].contiguous(), table)
    S.svdq_rope(heads, pos, table, out=heads)
    assert torch.equal(heads[-last:], want)
    S.svdq_check()
