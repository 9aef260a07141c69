"""Host-side refusals of the training entry points (CPU only): no handle, no GPU."""
import ctypes
import math

import pytest

from mixture_experts_layer_router_gb300 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def dims(batch=1, rows=64, cols=64, steps=5, coefs=None, eps=1e-7):
    return capi.latentmoe_muon_dims(batch, rows, cols, steps, coefs, eps)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), capi.ERR_INVALID_ARG), (dict(rows=0), capi.ERR_INVALID_ARG),
    (dict(cols=-1), capi.ERR_INVALID_ARG), (dict(steps=0), capi.ERR_INVALID_ARG),
    (dict(eps=0.0), capi.ERR_INVALID_ARG), (dict(eps=-1.0), capi.ERR_INVALID_ARG),
    (dict(eps=float("nan")), capi.ERR_INVALID_ARG), (dict(eps=float("inf")), capi.ERR_INVALID_ARG),
    (dict(rows=65537), capi.ERR_UNSUPPORTED), (dict(cols=1 << 40), capi.ERR_UNSUPPORTED),
    (dict(batch=65536), capi.ERR_UNSUPPORTED), (dict(steps=33), capi.ERR_UNSUPPORTED),
    (dict(batch=65535, rows=65536, cols=65536), capi.ERR_UNSUPPORTED),
])
def test_muon_create_refuses(lib, kw, code):
    h = ctypes.c_void_p(7)
    assert lib.latentmoe_muon_create(ctypes.byref(dims(**kw)), ctypes.byref(h)) == code
    assert h.value is None


@pytest.mark.parametrize("coefs", [[math.nan, 0, 0], [math.inf, 0, 0], [1e9, 0, 0],
                                   [4.0, 0.0, 0.0], [0.0, 0.0, 1.0], [0.01, -1.0, 0.0]])
def test_muon_create_refuses_coefficients(lib, coefs):
    """Not finite, growing without bound (4^32 in 32 steps), or without a linear
    term (X to the fifth power leaves the range that the scales are made for)."""
    arr = (ctypes.c_float * 96)(*(coefs * 32))
    h = ctypes.c_void_p(7)
    d = dims(steps=32, coefs=ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)))
    assert lib.latentmoe_muon_create(ctypes.byref(d), ctypes.byref(h)) == capi.ERR_INVALID_ARG
    assert h.value is None


def test_null_arguments(lib):
    h = ctypes.c_void_p(7)
    assert lib.latentmoe_muon_create(None, ctypes.byref(h)) == capi.ERR_INVALID_ARG
    assert h.value is None
    assert lib.latentmoe_muon_create(ctypes.byref(dims()), None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_orthogonalize(None, None, 0, None, None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_step(None, None, None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_set_sm_pairs(None, 0) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_get_status(None, None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_get_launch_count(None, None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_muon_last_cuda_error(None) == 0
    assert lib.latentmoe_muon_destroy(None) == capi.OK
    assert lib.latentmoe_balance_loss(None, None, 0, None, None, 1, 0, 1.0, 0.0, None, None,
                                      None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_balance_loss_from_stats(None, None, 1, 1.0, 0.0, None,
                                                 None) == capi.ERR_INVALID_ARG
    assert lib.latentmoe_router_backward(None, None, 0, None, None, None, None, None, 1, 0, 1.0,
                                         0.0, None, None, 0, None) == capi.ERR_INVALID_ARG


def test_binding_refuses_coefficient_lists(lib):
    with pytest.raises(ValueError):
        capi.Muon(8, 8, steps=5, coefs=[(1.0, 0.0, 0.0)] * 4)
    with pytest.raises(ValueError):
        capi.Muon(8, 8, steps=5, coefs=(1.0, 2.0))


class _Device:
    """A tensor as the binding sees one on the GPU: attributes and strides, no data."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("T,E", [(2, 1), (7, 16), (64, 13)])
def test_binding_refuses_rows_that_overlap(lib, T, E):
    """Expanded rows (stride 0, which the C entries read as E) and rows closer than E
    are refused before anything is launched; one row may have any stride."""
    import torch
    layer = object.__new__(capi.LatentMoE)
    layer.dims, layer.k, layer.handle = capi.latentmoe_dims(128, 128, E, 128, 0, T), 1, None
    idx = _Device(torch.zeros((T, 1), dtype=torch.int32))
    counts, tokens = _Device(torch.zeros((1, E), dtype=torch.int32)), _Device(
        torch.zeros(1, dtype=torch.int32))
    good = _Device(torch.zeros((T, E)))
    wide = _Device(torch.zeros((T, E + 3))[:, :E])
    assert layer._rows(good, "logits", T) == E
    assert layer._rows(wide, "logits", T) == E + 3
    one = torch.zeros((1, E))
    assert layer._rows(_Device(one.expand(1, E)), "logits", 1) == E
    bad = [_Device(one.expand(T, E))]
    if E > 1:
        bad.append(_Device(torch.zeros(T * E).as_strided((T, E), (E - 1, 1))))
    for x in bad:
        with pytest.raises(ValueError):
            layer.balance_loss(x, idx)
        with pytest.raises(ValueError):
            layer.router_backward(x, idx, counts, tokens)
        with pytest.raises(ValueError):
            layer.router_backward(good, idx, counts, tokens, out=x)
