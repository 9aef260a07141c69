"""Host-side refusals of the RMS norm, gated block and clipping entries (CPU only): addresses that
nothing reads, since every call here is refused before a launch."""
import ctypes
import math

import pytest
import torch

from mixture_experts_layer_router_gb300 import build, capi

INVALID, UNSUPPORTED = capi.ERR_INVALID_ARG, capi.ERR_UNSUPPORTED
A = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def norm(**kw):
    a = dict(x=A, weight=A, y=A, eps=1e-6)
    a.update(kw)
    return capi.latentmoe_norm(**a)


@pytest.mark.parametrize("kw,T,d,code", [
    (dict(x=None), 4, 64, INVALID), (dict(weight=None), 4, 64, INVALID),
    (dict(y=None), 4, 64, INVALID), (dict(codes=A), 4, 64, INVALID),
    (dict(codes=A, scales=A, scale_block=64), 4, 64, INVALID), (dict(sum=A), 4, 64, INVALID),
    (dict(x_dtype=2), 4, 64, INVALID), (dict(weight_dtype=-1), 4, 64, INVALID),
    (dict(y_dtype=7), 4, 64, INVALID), (dict(residual=A, residual_dtype=3), 4, 64, INVALID),
    (dict(eps=0.0), 4, 64, INVALID), (dict(eps=math.nan), 4, 64, INVALID),
    (dict(eps=math.inf), 4, 64, INVALID), (dict(eps=-1.0), 4, 64, INVALID),
    (dict(), 0, 64, INVALID), (dict(), -1, 64, INVALID), (dict(), 4, 0, INVALID),
    (dict(ld_x=63), 4, 64, INVALID), (dict(ld_y=-64), 4, 64, INVALID),
    (dict(residual=A, ld_residual=1), 4, 64, INVALID), (dict(ld_codes=5), 4, 64, INVALID),
    (dict(), 4, 16385, UNSUPPORTED), (dict(), 1 << 31, 64, UNSUPPORTED),
    (dict(x_dtype=1, residual=A), 4, 64, UNSUPPORTED), (dict(x=A + 1), 4, 64, UNSUPPORTED),
    (dict(x=A + 2, x_dtype=1), 4, 64, UNSUPPORTED), (dict(y=A + 2, y_dtype=1), 4, 64, UNSUPPORTED),
    (dict(weight=A + 1), 4, 64, UNSUPPORTED), (dict(rstd=A + 2), 4, 64, UNSUPPORTED),
    (dict(codes=A, scales=A + 1), 4, 64, UNSUPPORTED),
    (dict(residual=A + 2, residual_dtype=1), 4, 64, UNSUPPORTED),
])
def test_norm_refuses(lib, kw, T, d, code):
    assert lib.latentmoe_rms_norm(ctypes.byref(norm(**kw)), T, d, None) == code


def grad(**kw):
    a = dict(dy=A, s=A, weight=A, rstd=A, dx=A)
    a.update(kw)
    return capi.latentmoe_norm_grad(**a)


@pytest.mark.parametrize("kw,T,d,ws,size,code", [
    (dict(dy=None), 4, 64, A, 1 << 30, INVALID), (dict(s=None), 4, 64, A, 1 << 30, INVALID),
    (dict(weight=None), 4, 64, A, 1 << 30, INVALID), (dict(rstd=None), 4, 64, A, 1 << 30, INVALID),
    (dict(dx=None), 4, 64, A, 1 << 30, INVALID), (dict(dx16=A), 4, 64, A, 1 << 30, INVALID),
    (dict(dw=A), 4, 64, None, 1 << 30, INVALID), (dict(dw=A), 4, 64, A, 64 * 4 - 1, INVALID),
    (dict(s_dtype=9), 4, 64, A, 1 << 30, INVALID), (dict(ld_dx=8), 4, 64, A, 1 << 30, INVALID),
    (dict(), 0, 64, A, 1 << 30, INVALID), (dict(), 4, 20000, A, 1 << 30, UNSUPPORTED),
    (dict(dw=A), 4, 64, A + 8, 1 << 30, UNSUPPORTED), (dict(dy=A + 1), 4, 64, A, 1 << 30, UNSUPPORTED),
    (dict(d_sum=A + 2, s_dtype=1), 4, 64, A, 1 << 30, UNSUPPORTED),
])
def test_norm_backward_refuses(lib, kw, T, d, ws, size, code):
    assert lib.latentmoe_rms_norm_backward(ctypes.byref(grad(**kw)), T, d, ws, size, None) == code


def test_norm_null(lib):
    assert lib.latentmoe_rms_norm(None, 1, 1, None) == INVALID
    assert lib.latentmoe_rms_norm_backward(None, 1, 1, None, 0, None) == INVALID
    size = lib.latentmoe_rms_norm_backward_workspace
    assert size(0, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0
    assert size(4, 1024) >= 1024 * 4
    assert size(1 << 20, 1024) <= 256 * 32 * 1024 * 4


def table(*rows):
    return (capi.latentmoe_gradient * max(1, len(rows)))(*[capi.latentmoe_gradient(*r) for r in rows])


GOOD = (A, A, 100, 0)


@pytest.mark.parametrize("rows,code", [
    ([(None, A, 5, 0)], INVALID), ([(A, None, 5, 0)], INVALID), ([(A, A, -1, 0)], INVALID),
    ([(A, A, 5, 2)], INVALID), ([(A, A, 5, -1)], INVALID), ([(A + 1, A + 1, 5, 0)], UNSUPPORTED),
    ([(A + 2, A + 2, 5, 1)], UNSUPPORTED), ([(A, A + 1, 5, 0)], UNSUPPORTED),
    ([(A, A, 1 << 50, 0)], UNSUPPORTED),
    ([GOOD, GOOD], INVALID), ([(A, A, 100, 0), (A + 198, A + 198, 5, 0)], INVALID),
    ([(A, A + 2, 100, 0)], INVALID), ([(A, A + 4096, 100, 0), (A + 4096, A + 8192, 100, 0)], INVALID),
])
def test_clip_refuses(lib, rows, code):
    t = table(*rows)
    n = len(rows)
    assert lib.latentmoe_grad_clip(t, n, 1.0, 1e-6, A, A, 1 << 20, None) == code


def test_clip_refuses_numbers_and_scratch(lib):
    t = table(GOOD)
    call = lib.latentmoe_grad_clip
    for max_norm, eps in ((-1.0, 0.0), (math.nan, 0.0), (1.0, -1.0), (1.0, math.nan), (1.0, math.inf)):
        assert call(t, 1, max_norm, eps, A, A, 1 << 20, None) == INVALID
    assert call(t, -1, 1.0, 0.0, A, A, 1 << 20, None) == INVALID
    assert call(None, 1, 1.0, 0.0, A, A, 1 << 20, None) == INVALID
    assert call(t, 1, 1.0, 0.0, None, A, 1 << 20, None) == INVALID
    assert call(t, 1, 1.0, 0.0, A, None, 1 << 20, None) == INVALID
    assert call(t, 1, 1.0, 0.0, A, A, lib.latentmoe_grad_workspace(1) - 1, None) == INVALID
    assert call(t, 1, 1.0, 0.0, A, A + 8, 1 << 20, None) == UNSUPPORTED
    assert call(t, 1, 1.0, 0.0, A + 2, A, 1 << 20, None) == UNSUPPORTED
    assert lib.latentmoe_grad_norm(None, 1, A, A, 1 << 20, None) == INVALID
    assert lib.latentmoe_grad_norm(t, 1, A, A, 8, None) == INVALID
    assert lib.latentmoe_grad_workspace(-1) == 0
    assert lib.latentmoe_grad_workspace(1001) == 2 * lib.latentmoe_grad_workspace(1000)


def test_binding_refuses_host_tensors(lib):
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        capi.rms_norm(x, w)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        capi.rms_norm(x, w, quantize="row")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        capi.rms_norm_backward(x, x, w, torch.zeros(2))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        capi.clip_gradients([x], 1.0)
    with pytest.raises(ValueError):
        capi.gradient_norm([])


@pytest.mark.parametrize("dims,code", [
    ((0, 8, 1, 0), INVALID), ((8, 0, 1, 0), INVALID), ((8, 8, 0, 0), INVALID), ((-8, 8, 1, 0), INVALID),
    ((12, 8, 1, 0), UNSUPPORTED), ((8, 4, 1, 0), UNSUPPORTED), ((65544, 8, 1, 0), UNSUPPORTED),
    ((8, 1 << 40, 1, 0), UNSUPPORTED), ((8, 8, (1 << 22) + 1, 1), UNSUPPORTED),
])
def test_ffn_create_refuses(lib, dims, code):
    h = ctypes.c_void_p(7)
    d = capi.latentmoe_ffn_dims(*dims)
    assert lib.latentmoe_ffn_create(ctypes.byref(d), ctypes.byref(h)) == code
    assert h.value is None


def test_ffn_null(lib):
    h = ctypes.c_void_p(7)
    assert lib.latentmoe_ffn_create(None, ctypes.byref(h)) == INVALID
    assert h.value is None
    assert lib.latentmoe_ffn_create(ctypes.byref(capi.latentmoe_ffn_dims(8, 8, 1, 0)), None) == INVALID
    assert lib.latentmoe_ffn_forward(None, None, None, 0, None, 0, None, None, 1, None) == INVALID
    assert lib.latentmoe_ffn_backward(None, None, None, 1, None) == INVALID
    assert lib.latentmoe_ffn_set_sm_pairs(None, 0) == INVALID
    assert lib.latentmoe_ffn_get_status(None, None) == INVALID
    assert lib.latentmoe_ffn_get_launch_count(None, None) == INVALID
    assert lib.latentmoe_ffn_last_cuda_error(None) == 0
    assert lib.latentmoe_ffn_destroy(None) == capi.OK
