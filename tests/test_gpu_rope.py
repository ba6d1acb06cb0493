"""Rotary positions over several axes on the GPU, against the 64-bit oracle
within counted roundings."""
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


def check(X, x, pos, table, interleaved, inverse, out=None):
    Y = S.svdq_rope(X, pos.cuda(), table, interleaved, inverse, out=out)
    y, bound = B.rope(B.np64(x), B.np64(pos), table.axis_dims, B.np64(table.freqs), interleaved, inverse)
    R = sum(table.axis_dims)
    B.within(Y, y, bound + B.rounding(y, X.dtype), "Y")
    assert torch.equal(Y[..., R:].cpu(), x[..., R:])      # what is not turned is copied
    return Y


# heads of whole and partial rotation, sections that end inside a vector, odd pair counts, one token, many tokens
@pytest.mark.parametrize("T,H,D,dims", [(1, 1, 2, (2,)), (7, 40, 80, (16, 32, 32)), (3, 2, 128, (16, 56, 56)),
                                        (50, 3, 128, (44, 42, 42)), (9, 5, 96, (10, 14)), (4, 64, 64, (2, 2, 2, 2)),
                                        (700, 6, 48, (8, 20, 20)), (2, 3, 512, (512,)), (5, 2, 18, (6, 6, 4)),
                                        (33, 7, 256, (32, 48, 48))])
@pytest.mark.parametrize("dtype", [BF, FP16, FP32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_turns(T, H, D, dims, dtype, interleaved):
    g = torch.Generator().manual_seed(T + H + D)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.randint(0, 300, (T, len(dims)), generator=g, dtype=torch.int32)
    table = S.svdq_rope_table(dims)
    check(x.cuda(), x, pos, table, interleaved, False)
    check(x.cuda(), x, pos.float() * 0.37 - 20, table, interleaved, True)


@pytest.mark.parametrize("pos", [torch.int32, FP32])
def test_far_positions_keep_their_angle(pos):
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(0))
    at = torch.tensor([[0, 1], [100000, 7], [-5, 16777216], [2000000, -1000000], [1, 0], [123456, 654321]])
    if pos == torch.int32:
        at[0, 0] = 2 ** 31 - 1
    check(x.cuda(), x, at.to(pos), S.svdq_rope_table((32, 32)), True, False)


@pytest.mark.parametrize("dtype", [BF, FP32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,dims", [(64, (16, 24, 24)), (20, (8, 8))])
def test_heads_inside_a_merged_projection_and_in_place(dtype, interleaved, D, dims):
    T, H = 40, 3
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(T, 3 * H, D, generator=g).to(dtype)
    pos = torch.randint(0, 64, (T, len(dims)), generator=g, dtype=torch.int32)
    table = S.svdq_rope_table(dims)
    dev = qkv.cuda()
    want = check(dev[:, :2 * H], qkv[:, :2 * H], pos, table, interleaved, False)
    S.svdq_rope(dev[:, :2 * H], pos.cuda(), table, interleaved, out=dev[:, :2 * H])
    assert torch.equal(dev[:, :2 * H], want) and torch.equal(dev[:, 2 * H:].cpu(), qkv[:, 2 * H:])


def test_heads_ahead_of_tokens_and_repeated_heads():
    T, H, D = 30, 4, 32
    g = torch.Generator().manual_seed(2)
    pos = torch.randint(0, 64, (T, 2), generator=g, dtype=torch.int32)
    table = S.svdq_rope_table((16, 16))
    x = torch.randn(H, T, D, generator=g).to(BF)
    X = x.cuda().transpose(0, 1)
    out = torch.empty(H, T, D, dtype=BF, device="cuda").transpose(0, 1)
    check(X, x.transpose(0, 1), pos, table, True, False, out=out)
    one = torch.randn(T, 1, D, generator=g).to(BF)          # a shared key head, repeated for its queries
    check(one.cuda().expand(T, H, D), one.expand(T, H, D), pos, table, True, False)


def test_a_batch_shares_its_positions():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(36, 2, 16, generator=g).to(FP16)
    pos = torch.randint(0, 64, (12, 2), generator=g, dtype=torch.int32)
    check(x.cuda(), x, pos, S.svdq_rope_table((8, 8)), False, False)


def test_gradient():
    """<rope(x), dy> against differences, and rope followed by its inverse gives x back."""
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(3, 2, 12, generator=g), torch.randn(3, 2, 12, generator=g)
    pos = torch.randint(0, 64, (3, 2), generator=g, dtype=torch.int32)
    table = S.svdq_rope_table((4, 6))
    for interleaved in (True, False):
        dX = S.svdq_rope(dy.cuda(), pos.cuda(), table, interleaved, inverse=True)
        num = np.zeros(x.shape)
        for i in np.ndindex(num.shape):
            e = np.zeros(x.shape)
            e[i] = 1.0                                      # the map is linear: a unit step is exact
            num[i] = (B.rope(e, B.np64(pos), (4, 6), B.np64(table.freqs), interleaved, False)[0] * B.np64(dy)).sum()
        np.testing.assert_allclose(B.np64(dX), num, rtol=0, atol=16 * B.U * 8)
        back = S.svdq_rope(S.svdq_rope(x.cuda(), pos.cuda(), table, interleaved), pos.cuda(), table, interleaved, True)
        np.testing.assert_allclose(B.np64(back), B.np64(x), rtol=0, atol=32 * B.U * 8)


def test_nothing_to_turn():
    table = S.svdq_rope_table((8,))
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    assert S.svdq_rope(torch.empty(0, 3, 8, device="cuda"), pos, table).shape == (0, 3, 8)
    assert S.svdq_rope(torch.empty(2, 0, 8, device="cuda"), pos, table).shape == (2, 0, 8)


def test_replayed_graph():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(64, 4, 32, generator=g).cuda()
    pos = torch.randint(0, 64, (64, 2), generator=g, dtype=torch.int32).cuda()
    table = S.svdq_rope_table((16, 16))
    S.svdq_rope(x, pos, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = S.svdq_rope(x, pos, table)
    x.neg_()
    pos.add_(3)
    graph.replay()
    assert torch.equal(y, S.svdq_rope(x, pos, table))
