"""Host-side checks of the operators around the 4-bit linear layer (no GPU):
shapes, types, strides, null and misaligned pointers are refused with the
documented status before a device is touched, and the binding refuses tensors
that do not fit."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import block_oracle as O
from w4a4_diffusion_model_b200 import build as B
from w4a4_diffusion_model_b200 import svdq as S

GOOD, BAD = 1 << 20, (1 << 20) + 8
ARG, SHAPE, ALIGN, SMALL, NODEV = 1, 2, 3, 4, 5
BF, FP16, FP32, I32 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    B.build()
    return S.load()


def quant(lib, M=4, K=64, dt=BF, x=GOOD, ld=64, mult=None, q=GOOD, s=GOOD):
    return lib.svdq_int8_quantize_act(M, K, dt, x, ld, mult, q, s, None)


def linear(lib, M=4, K=64, N=8, qx=GOOD, sx=GOOD, qw=GOOD, sw=GOOD, b=None, dt=BF, y=GOOD, ld=8):
    return lib.svdq_int8_linear(M, K, N, qx, sx, qw, sw, b, dt, y, ld, None)


def norm(lib, M=4, C=64, dt=BF, wt=BF, x=GOOD, ld=64, w=GOOD, b=GOOD, rows=0, eps=1e-6, flags=0, y=GOOD, ldy=64,
         mean=None, rstd=None):
    return lib.svdq_layernorm(M, C, dt, wt, x, ld, w, b, rows, eps, flags, y, ldy, mean, rstd, None)


def backward(lib, M=4, C=64, dt=BF, wt=BF, dy=GOOD, lddy=64, x=GOOD, ld=64, w=GOOD, mean=GOOD, rstd=GOOD, rows=0,
             flags=0, dx=GOOD, lddx=64, dw=None, db=None, ws=None, wsb=0):
    return lib.svdq_layernorm_backward(M, C, dt, wt, dy, lddy, x, ld, w, mean, rstd, rows, flags, dx, lddx, dw, db, ws,
                                       wsb, None)


def rope(lib, T=4, H=2, D=16, dt=BF, x=GOOD, xt=32, xh=16, y=GOOD, yt=32, yh=16, pos=GOOD, pt=I32, rows=4,
         dims=(8, 8), freqs=GOOD, flags=0):
    return lib.svdq_rope(T, H, D, dt, x, xt, xh, y, yt, yh, pos, pt, rows, len(dims), (ctypes.c_int32 * 8)(*dims),
                         freqs, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=8), SHAPE), (dict(K=24), SHAPE), (dict(K=131088), SHAPE), (dict(M=(1 << 30) + 1), SHAPE),
    (dict(dt=3), ARG), (dict(dt=-1), ARG), (dict(x=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG),
    (dict(ld=63), ARG), (dict(ld=-64), ARG), (dict(ld=68), ALIGN), (dict(x=BAD), ALIGN), (dict(mult=BAD), ALIGN),
    (dict(q=BAD), ALIGN), (dict(s=BAD), ALIGN)])
def test_quantizer_refusals(lib, kw, status):
    assert quant(lib, **kw) == status
    assert lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=40), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 24) + 1), SHAPE), (dict(dt=3), ARG),
    (dict(qx=None), ARG), (dict(sx=None), ARG), (dict(qw=None), ARG), (dict(sw=None), ARG), (dict(y=None), ARG),
    (dict(ld=7), ARG), (dict(b=BAD), ALIGN), (dict(y=BAD), ALIGN), (dict(qw=BAD), ALIGN)])
def test_product_refusals(lib, kw, status):
    assert linear(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(C=0), SHAPE), (dict(C=16385, ld=16385, ldy=16385), SHAPE), (dict(dt=3), ARG),
    (dict(wt=FP16), ARG), (dict(rows=-1), ARG), (dict(flags=2), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(ldy=72), ARG), (dict(x=None), ARG), (dict(y=None), ARG), (dict(ld=63), ARG), (dict(ldy=63), ARG),
    (dict(x=BAD), ALIGN), (dict(mean=BAD), ALIGN), (dict(rstd=BAD), ALIGN), (dict(w=BAD), ALIGN), (dict(b=BAD), ALIGN)])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_norm_into_codes_refusals(lib):
    call = lambda C=64, q=GOOD, s=GOOD, lam=None: lib.svdq_int8_layernorm_quantize(  # noqa: E731
        4, C, BF, BF, GOOD, 64, None, None, 0, 1e-6, 0, lam, q, s, None)
    assert call(C=40) == SHAPE and call(q=None) == ARG and call(s=None) == ARG and call(lam=BAD) == ALIGN


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG), (dict(dx=None), ARG), (dict(lddy=60), ARG),
    (dict(lddx=60), ARG), (dict(lddx=72), ARG), (dict(dx=BAD), ALIGN), (dict(flags=4), ARG), (dict(wt=1), ARG), (dict(C=20000), SHAPE),
    (dict(M=5000, dw=GOOD), SMALL), (dict(M=5000, db=GOOD, ws=GOOD, wsb=64), SMALL)])
def test_backward_refusals(lib, kw, status):
    assert backward(lib, **kw) == status


def test_backward_workspace(lib):
    assert S.svdq_layernorm_backward_workspace(0, 64) == 0
    assert S.svdq_layernorm_backward_workspace(1, 64) == 0          # one chunk of rows: nothing to join
    many = S.svdq_layernorm_backward_workspace(9216, 4096, 4608)
    assert many > 0 and many % (2 * 2 * 4096 * 4) == 0
    assert S.svdq_layernorm_backward_workspace(9216, 64, 1) == 0    # a group per row: each block owns its rows
    with pytest.raises(S.SvdqError):
        S.svdq_layernorm_backward_workspace(4, 20000)
    assert lib.svdq_layernorm_backward_workspace(4, 64, 0, None) == ARG


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(D=15), SHAPE), (dict(D=514), SHAPE), (dict(H=-1), SHAPE), (dict(dt=3), ARG),
    (dict(pt=0), ARG), (dict(flags=4), ARG), (dict(dims=()), ARG), (dict(dims=(8, 7)), ARG), (dict(dims=(8, 0)), ARG),
    (dict(dims=(8, 10)), ARG), (dict(x=None), ARG), (dict(y=None), ARG), (dict(pos=None), ARG), (dict(freqs=None), ARG),
    (dict(rows=0), ARG), (dict(rows=3), ARG), (dict(xt=-32), ARG), (dict(y=BAD), ALIGN), (dict(pos=BAD), ALIGN),
    (dict(yt=16, yh=16), ARG), (dict(yh=8), ARG), (dict(xt=64), ARG), (dict(x=BAD), ALIGN)])
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device_is_reported(lib):
    for call in (quant, linear, norm, rope, backward):
        assert call(lib) == NODEV


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: S.svdq_int8_quantize_act(x), lambda: S.svdq_layernorm(x),
                 lambda: S.svdq_int8_prepare_weights(x), lambda: S.svdq_int8_layernorm_quantize(x),
                 lambda: S.svdq_layernorm_backward(x, x, None, x[:, 0], x[:, 0]),
                 lambda: S.svdq_rope(x.view(4, 2, 32), torch.zeros(4, 1), S.svdq_rope_table((32,), device="cpu"))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_rope_table():
    t = S.svdq_rope_table((16, 8), theta=100.0, device="cpu")
    assert t.freqs.dtype == torch.float64 and t.freqs.shape == (12,)
    np.testing.assert_allclose(t.freqs[:8].numpy(), 100.0 ** (-np.arange(0, 16, 2) / 16), rtol=1e-15)
    np.testing.assert_allclose(t.freqs[8:].numpy(), 100.0 ** (-np.arange(0, 8, 2) / 8), rtol=1e-15)
    with pytest.raises(ValueError):
        S.svdq_rope_table((16, 7), device="cpu")
    with pytest.raises(ValueError):
        S.RopeTable((16,), torch.zeros(8))


def test_oracle_codes_are_the_nearest():
    """The tests' own oracle against every code, by distance."""
    x = np.random.default_rng(0).normal(size=(3, 32)).astype(np.float32)
    q, s = O.int8_codes(x)
    for r in range(3):
        d = np.abs(x[r].astype(np.float64)[:, None] / float(s[r]) - np.arange(-127, 128))
        np.testing.assert_array_equal(q[r], d.argmin(1) - 127)
    assert np.abs(q).max() == 127


# rows around the limits of the few-rows form and past them; affine, and groups that share the blocks
@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls' pointers are made up: they must end at the missing device")
@pytest.mark.parametrize("M,rows", [(1, 0), (257, 0), (401, 0), (593, 0), (2000, 0), (70000, 0), (2000, 500), (2000, 7)])
def test_queried_workspace_serves_every_type_and_layout(lib, M, rows):
    """The query names neither type nor strides, so its answer has to do for each: 16-bit and fp32 rows of every width,
    dense and off 16-byte boundaries."""
    need = ctypes.c_size_t()
    refused = []
    for C in range(1, 16385):
        assert lib.svdq_layernorm_backward_workspace(M, C, rows, ctypes.byref(need)) == 0
        for dt in (BF, FP16, FP32):
            for ld in (C, C + 1):
                status = backward(lib, M=M, C=C, dt=dt, wt=dt, lddy=ld, ld=ld, lddx=ld, rows=rows, dw=GOOD, db=GOOD,
                                  ws=GOOD if need.value else None, wsb=need.value)
                if status != NODEV:
                    refused.append((C, dt, ld, status))
    assert not refused, f"{len(refused)} calls refused, the first {refused[:3]}"


def test_the_documented_codes_cannot_leave_int32(lib):
    """The extremes that the header allows, against int32's range: -127 to 127 on both sides at the largest K that is
    taken, -128 on one side, and -128 on both below the K it names."""
    assert linear(lib, K=131088) == SHAPE
    with open(os.path.join(B.ROOT, "include", "svdq.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    both = re.search(r"-128 too in Qx or in Qw, and in both where K < (\d+)", text)
    assert both, "codes of -128 need a limit on K"
    assert 127 * 127 * 131072 < 2 ** 31 and 128 * 127 * 131072 < 2 ** 31
    assert 128 * 128 * (int(both.group(1)) - 16) < 2 ** 31 <= 128 * 128 * int(both.group(1))


def test_the_scale_factor_is_a_sixteenth_of_a_step_off():
    """fp32(1/127) = (1/127) (1 - 2^-28), in whole numbers; and what the oracle's scales make of it."""
    c = float(np.float32(1) / np.float32(127))
    assert 127 * int(c * 2 ** 30) * 2 ** 5 == 2 ** 35 - 2 ** 7 and int(c * 2 ** 30) / 2 ** 30 == c
    x = np.random.default_rng(3).normal(size=(20000, 16)).astype(np.float32)
    q, s = O.int8_codes(x)
    top = np.abs(x.astype(np.float64)).max(1)
    assert (np.abs(s - top / 127) <= (0.5 + 1 / 16) * np.spacing(s)).all()
    off = 127 * (2.0 ** -24 + 2.0 ** -28) * (1 + 2.0 ** -20)
    assert (np.abs(q - 127 * x / top[:, None]) <= 0.5 + off).all()
