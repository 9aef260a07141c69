"""ctypes binding of liblatentmoe.so (include/latentmoe.h), same names.

Argument marshalling only: every step of the layer, of the training operators
(balance loss, router backward, Muon) and of the block around it (RMS norm,
gated feed-forward block, gradient clipping) runs in the library's CUDA kernels. PyTorch provides device memory (``tensor.data_ptr()``) and
streams (``torch.cuda.current_stream().cuda_stream``). There is no fallback:
``load()`` raises if the library is missing or cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional  # noqa: F401

_PKG = os.path.dirname(os.path.abspath(__file__))
# LATENTMOE_LIB names another build of the same library (the bounds-checked
# debug build, _build/bounds/liblatentmoe.so); there is no other fallback
LIB_PATH = os.environ.get("LATENTMOE_LIB") or os.path.join(_PKG, "_build", "liblatentmoe.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_NOT_LOADED = -3
ERR_CUDA = -4
ERR_TIMEOUT = -5
ERR_DEVICE_STATUS = -6
ERR_OUT_OF_MEMORY = -7

RENORM = 1
ROUTER_BIAS = 2
OUT_FP32 = 4
SELECT_BIAS = 8
FP8_EXPERTS = 16
FP8_DENSE = 32
FP8_TENSORS = 5  # scaled activations: z, h, x, c, shared hidden

BF16 = 0  # element types of a matrix update
FP32 = 1

STATUS_TIMEOUT = 1
STATUS_BAD_EXPERT = 2
STATUS_ROUNDS = 4
STATUS_BOUNDS = 8

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64


class latentmoe_dims(ctypes.Structure):
    _fields_ = [("hidden", _i64), ("latent", _i64), ("num_experts", _i64),
                ("ffn", _i64), ("shared_ffn", _i64), ("max_tokens", _i64)]


class latentmoe_weights(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in
                ("w_r", "b_r", "w_dn", "w_g", "w_u", "w_d", "w_up", "w_gs", "w_us", "w_ds")]


class latentmoe_balance_stats(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in ("counts", "prob_sum", "z_sum", "tokens")]


class latentmoe_muon_dims(ctypes.Structure):
    _fields_ = [("batch", _i64), ("rows", _i64), ("cols", _i64), ("steps", _i64),
                ("coefs", ctypes.POINTER(ctypes.c_float)), ("eps", ctypes.c_float)]


class latentmoe_muon_update(ctypes.Structure):
    _fields_ = [("g", _c_void_p), ("momentum", _c_void_p), ("w", _c_void_p),
                ("g_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("nesterov", ctypes.c_int32), ("lr", ctypes.c_float),
                ("momentum_coef", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float)]


class latentmoe_ffn_dims(ctypes.Structure):
    _fields_ = [("hidden", _i64), ("ffn", _i64), ("max_tokens", _i64), ("training", ctypes.c_int32)]


class latentmoe_ffn_weights(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in ("w_g", "w_u", "w_d")]


class latentmoe_ffn_grad(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in ("dy", "x", "gate", "up", "dx", "dw_g", "dw_u", "dw_d")] + \
        [(n, _i64) for n in ("ld_dy", "ld_x", "ld_dx")] + \
        [(n, ctypes.c_int32) for n in ("dw_dtype", "accumulate")]


class latentmoe_norm(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in
                ("x", "residual", "weight", "sum", "y", "codes", "scales", "rstd")] + \
        [(n, _i64) for n in ("ld_x", "ld_residual", "ld_sum", "ld_y", "ld_codes")] + \
        [(n, ctypes.c_int32) for n in ("x_dtype", "residual_dtype", "weight_dtype", "y_dtype",
                                       "scale_block")] + [("eps", ctypes.c_float)]


class latentmoe_norm_grad(ctypes.Structure):
    _fields_ = [(n, _c_void_p) for n in
                ("dy", "s", "weight", "rstd", "d_sum", "dx", "dx16", "dw")] + \
        [(n, _i64) for n in ("ld_dy", "ld_s", "ld_d_sum", "ld_dx", "ld_dx16")] + \
        [(n, ctypes.c_int32) for n in ("dy_dtype", "s_dtype", "weight_dtype")]


class latentmoe_gradient(ctypes.Structure):
    _fields_ = [("g", _c_void_p), ("out", _c_void_p), ("n", _i64), ("dtype", _i64)]


# name -> (restype, argtypes)
SIGNATURES = {
    "latentmoe_create": (ctypes.c_int, [ctypes.POINTER(latentmoe_dims), ctypes.c_int,
                                        ctypes.c_uint32, ctypes.POINTER(_c_void_p)]),
    "latentmoe_load_weights": (ctypes.c_int, [_c_void_p, ctypes.POINTER(latentmoe_weights),
                                                _c_void_p]),
    "latentmoe_forward": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p]),
    "latentmoe_forward_routed": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                _c_void_p, _i64, _c_void_p]),
    "latentmoe_forward_host": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p]),
    "latentmoe_forward_host_async": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64,
                                                    _c_void_p]),
    "latentmoe_host_wait": (ctypes.c_int, [_c_void_p]),
    "latentmoe_destroy": (ctypes.c_int, [_c_void_p]),
    "latentmoe_route_from_logits": (ctypes.c_int, [_c_void_p, _c_void_p, _i64] + [_c_void_p] * 7),
    "latentmoe_route_from_logits_static": (ctypes.c_int, [_c_void_p, _i64, _i64, ctypes.c_int,
                                                          ctypes.c_uint32] + [_c_void_p] * 7),
    "latentmoe_lbl_stats": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "latentmoe_get_routing": (ctypes.c_int, [_c_void_p] + [_c_void_p] * 7 + [_c_void_p]),
    "latentmoe_get_status": (ctypes.c_int, [_c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "latentmoe_set_profiling": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_get_stage_times": (ctypes.c_int, [_c_void_p, ctypes.c_int,
                                                 ctypes.POINTER(ctypes.c_float), ctypes.c_int]),
    "latentmoe_num_stages": (ctypes.c_int, []),
    "latentmoe_stage_name": (ctypes.c_char_p, [ctypes.c_int]),
    "latentmoe_get_launch_count": (ctypes.c_int, [_c_void_p, ctypes.POINTER(_i64)]),
    "latentmoe_set_pdl": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_set_sm_pairs": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_set_expert_fusion": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_set_capacity": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64]),
    "latentmoe_get_rounds": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.POINTER(ctypes.c_int32)]),
    "latentmoe_last_cuda_error": (ctypes.c_int, [_c_void_p]),
    "latentmoe_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "latentmoe_debug_gemm": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64,
                                            ctypes.c_int, _c_void_p]),
    "latentmoe_debug_grouped_gemm": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                    _i64, _i64, _i64, _i64, ctypes.c_int,
                                                    _c_void_p]),
    "latentmoe_get_fp8_state": (ctypes.c_int, [_c_void_p, ctypes.POINTER(ctypes.c_float),
                                               ctypes.POINTER(ctypes.c_float),
                                               ctypes.POINTER(_i64)]),
    "latentmoe_get_fp8_codes": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "latentmoe_set_fp8_scales": (ctypes.c_int, [_c_void_p, ctypes.POINTER(ctypes.c_float)]),
    "latentmoe_get_fp8_dense_codes": (ctypes.c_int, [_c_void_p] * 5),
    "latentmoe_get_fp8_weight_scales": (ctypes.c_int, [_c_void_p,
                                                       ctypes.POINTER(ctypes.c_float)]),
    "latentmoe_quantize_e4m3": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64, _c_void_p,
                                               _c_void_p, _c_void_p]),
    "latentmoe_debug_grouped_gemm_e4m3": (ctypes.c_int, [_c_void_p] * 6 + [_i64] * 4 +
                                          [ctypes.c_int, _c_void_p]),
    "latentmoe_balance_loss": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p,
                                              _i64, _i64, ctypes.c_float, ctypes.c_float,
                                              ctypes.POINTER(latentmoe_balance_stats), _c_void_p,
                                              _c_void_p]),
    "latentmoe_balance_loss_from_stats": (ctypes.c_int,
                                          [_c_void_p, ctypes.POINTER(latentmoe_balance_stats),
                                           _i64, ctypes.c_float, ctypes.c_float, _c_void_p,
                                           _c_void_p]),
    "latentmoe_router_backward": (ctypes.c_int, [_c_void_p, _c_void_p, _i64] + [_c_void_p] * 5 +
                                  [_i64, _i64, ctypes.c_float, ctypes.c_float, _c_void_p,
                                   _c_void_p, _i64, _c_void_p]),
    "latentmoe_muon_create": (ctypes.c_int, [ctypes.POINTER(latentmoe_muon_dims),
                                             ctypes.POINTER(_c_void_p)]),
    "latentmoe_muon_orthogonalize": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _c_void_p,
                                                    _c_void_p]),
    "latentmoe_muon_step": (ctypes.c_int, [_c_void_p, ctypes.POINTER(latentmoe_muon_update),
                                           _c_void_p]),
    "latentmoe_muon_set_sm_pairs": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_muon_get_status": (ctypes.c_int, [_c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "latentmoe_muon_get_launch_count": (ctypes.c_int, [_c_void_p, ctypes.POINTER(_i64)]),
    "latentmoe_muon_last_cuda_error": (ctypes.c_int, [_c_void_p]),
    "latentmoe_muon_destroy": (ctypes.c_int, [_c_void_p]),
    "latentmoe_ffn_create": (ctypes.c_int, [ctypes.POINTER(latentmoe_ffn_dims),
                                            ctypes.POINTER(_c_void_p)]),
    "latentmoe_ffn_forward": (ctypes.c_int, [_c_void_p, ctypes.POINTER(latentmoe_ffn_weights),
                                             _c_void_p, _i64, _c_void_p, _i64, _c_void_p, _c_void_p,
                                             _i64, _c_void_p]),
    "latentmoe_ffn_backward": (ctypes.c_int, [_c_void_p, ctypes.POINTER(latentmoe_ffn_weights),
                                              ctypes.POINTER(latentmoe_ffn_grad), _i64, _c_void_p]),
    "latentmoe_ffn_set_sm_pairs": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "latentmoe_ffn_get_status": (ctypes.c_int, [_c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "latentmoe_ffn_get_launch_count": (ctypes.c_int, [_c_void_p, ctypes.POINTER(_i64)]),
    "latentmoe_ffn_last_cuda_error": (ctypes.c_int, [_c_void_p]),
    "latentmoe_ffn_destroy": (ctypes.c_int, [_c_void_p]),
    "latentmoe_rms_norm": (ctypes.c_int, [ctypes.POINTER(latentmoe_norm), _i64, _i64,
                                          _c_void_p]),
    "latentmoe_rms_norm_backward": (ctypes.c_int, [ctypes.POINTER(latentmoe_norm_grad), _i64, _i64,
                                                   _c_void_p, ctypes.c_size_t, _c_void_p]),
    "latentmoe_rms_norm_backward_workspace": (ctypes.c_size_t, [_i64, _i64]),
    "latentmoe_grad_norm": (ctypes.c_int, [_c_void_p, _i64, _c_void_p, _c_void_p,
                                           ctypes.c_size_t, _c_void_p]),
    "latentmoe_grad_clip": (ctypes.c_int, [_c_void_p, _i64, ctypes.c_double, ctypes.c_double,
                                           _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "latentmoe_grad_workspace": (ctypes.c_size_t, [_i64]),
    "latentmoe_debug_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32)]),
    "latentmoe_debug_wait_timeout": (ctypes.c_int, [ctypes.c_uint64,
                                                    ctypes.POINTER(ctypes.c_uint32)]),
}

_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once) and declare every entry point."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -m mixture_experts_layer_router_gb300.build)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class LatentMoEError(RuntimeError):
    def __init__(self, code: int, what: str, cuda_error: int = 0):
        self.code = code
        self.cuda_error = cuda_error
        msg = load().latentmoe_strerror(code).decode()
        extra = f", cudaError {cuda_error}" if cuda_error else ""
        super().__init__(f"{what}: {msg} ({code}{extra})")


def check(code: int, what: str, handle=None) -> None:
    if code != OK:
        cuda = load().latentmoe_last_cuda_error(handle) if handle is not None else 0
        raise LatentMoEError(code, what, cuda)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _on_stream(stream, call, *args, **kw):
    """call(..., stream=None) with ``stream`` as the current one, so that the outputs
    it allocates are that stream's: memory whose last use on the caller's current
    stream has not ended yet is not handed out to them. Inputs made on another
    stream are the caller's to wait for and to record, as everywhere in torch."""
    import torch
    with torch.cuda.stream(stream):
        return call(*args, **kw)


_raw_stream = None  # () -> handle of the current stream


def _stream(stream) -> Optional[int]:
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        # without building a Stream object (3 us, a fifth of a small call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        if raw is None or dev is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            torch.cuda.current_stream()  # CUDA is initialised from here on
            _raw_stream = lambda: raw(dev())  # noqa: E731
    return _raw_stream()


class LatentMoE:
    """A handle on one layer. ``load_weights`` takes a dict as made by
    ``synth.make_weights`` (device bf16 tensors, ``b_r`` fp32 or None); the
    library copies them, so the caller may drop its tensors afterwards."""

    def __init__(self, d: int, l: int, E: int, k: int, F: int, Fs: int = 0,
                 max_tokens: int = 1, renorm: bool = False, router_bias: bool = False,
                 out_fp32: bool = False, select_bias: bool = False, fp8: bool = False,
                 fp8_dense: bool = False):
        lib = load()
        self.dims = latentmoe_dims(d, l, E, F, Fs, max_tokens)
        self.k = k
        self.flags = (RENORM if renorm else 0) | (ROUTER_BIAS if router_bias else 0) | \
            (OUT_FP32 if out_fp32 else 0) | (SELECT_BIAS if select_bias else 0) | \
            (FP8_EXPERTS if fp8 else 0) | (FP8_DENSE if fp8_dense else 0)
        h = _c_void_p()
        check(lib.latentmoe_create(ctypes.byref(self.dims), k, self.flags, ctypes.byref(h)),
              "latentmoe_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            load().latentmoe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_weights(self, w: Dict[str, object], stream=None) -> None:
        lw = latentmoe_weights(*(_ptr(w.get(n)) for n in
                                 ("w_r", "b_r", "w_dn", "w_g", "w_u", "w_d", "w_up",
                                  "w_gs", "w_us", "w_ds")))
        check(load().latentmoe_load_weights(self.handle, ctypes.byref(lw), _stream(stream)),
              "latentmoe_load_weights", self.handle)

    def forward(self, x, out=None, stream=None):
        import torch
        T = x.shape[0]
        if out is None:
            dt = torch.float32 if self.flags & OUT_FP32 else torch.bfloat16
            out = torch.empty((T, self.dims.hidden), dtype=dt, device=x.device)
        check(load().latentmoe_forward(self.handle, x.data_ptr(), out.data_ptr(), T,
                                       _stream(stream)), "latentmoe_forward", self.handle)
        return out

    def forward_routed(self, x, idx, gates=None, out=None, stream=None):
        """Router replay: idx [T, k] int32 (and optionally gates [T, k] fp32) given."""
        import torch
        T = x.shape[0]
        if out is None:
            dt = torch.float32 if self.flags & OUT_FP32 else torch.bfloat16
            out = torch.empty((T, self.dims.hidden), dtype=dt, device=x.device)
        check(load().latentmoe_forward_routed(self.handle, x.data_ptr(), idx.data_ptr(),
                                              _ptr(gates), out.data_ptr(), T, _stream(stream)),
              "latentmoe_forward_routed", self.handle)
        return out

    def forward_host(self, x_host, out_host, stream=None):
        check(load().latentmoe_forward_host(self.handle, x_host.data_ptr(), out_host.data_ptr(),
                                            x_host.shape[0], _stream(stream)),
              "latentmoe_forward_host")
        return out_host

    def forward_host_async(self, x_host, out_host, stream=None):
        """Pipelined host-buffer forward: returns at once; x_host must stay
        unchanged and out_host unread until host_wait()."""
        check(load().latentmoe_forward_host_async(self.handle, x_host.data_ptr(),
                                                  out_host.data_ptr(), x_host.shape[0],
                                                  _stream(stream)),
              "latentmoe_forward_host_async")
        return out_host

    def host_wait(self) -> None:
        check(load().latentmoe_host_wait(self.handle), "latentmoe_host_wait")

    def route_from_logits(self, logits, stream=None):
        import torch
        T, E = logits.shape
        dev = logits.device
        k = self.k
        out = {
            "idx": torch.empty((T, k), dtype=torch.int32, device=dev),
            "gates": torch.empty((T, k), dtype=torch.float32, device=dev),
            "counts": torch.empty((E,), dtype=torch.int32, device=dev),
            "offsets": torch.empty((E + 1,), dtype=torch.int32, device=dev),
            "perm": torch.empty((T * k,), dtype=torch.int32, device=dev),
            "pos": torch.empty((T, k), dtype=torch.int32, device=dev),
        }
        check(load().latentmoe_route_from_logits(
            self.handle, logits.data_ptr(), T, out["idx"].data_ptr(), out["gates"].data_ptr(),
            out["counts"].data_ptr(), out["offsets"].data_ptr(), out["perm"].data_ptr(),
            out["pos"].data_ptr(), _stream(stream)), "latentmoe_route_from_logits")
        return out

    def get_routing(self, T: int, device, stream=None):
        import torch
        E, k = self.dims.num_experts, self.k
        out = {
            "logits": torch.empty((T, E), dtype=torch.float32, device=device),
            "idx": torch.empty((T, k), dtype=torch.int32, device=device),
            "gates": torch.empty((T, k), dtype=torch.float32, device=device),
            "counts": torch.empty((E,), dtype=torch.int32, device=device),
            "offsets": torch.empty((E + 1,), dtype=torch.int32, device=device),
            "perm": torch.empty((T * k,), dtype=torch.int32, device=device),
            "pos": torch.empty((T, k), dtype=torch.int32, device=device),
        }
        check(load().latentmoe_get_routing(
            self.handle, *(out[n].data_ptr() for n in
                           ("logits", "idx", "gates", "counts", "offsets", "perm", "pos")),
            _stream(stream)), "latentmoe_get_routing")
        return out

    def lbl_stats(self, device, stream=None):
        """(prob_sum [E] fp32, counts [E] int32) of the last forward."""
        import torch
        E = self.dims.num_experts
        ps = torch.empty((E,), dtype=torch.float32, device=device)
        cn = torch.empty((E,), dtype=torch.int32, device=device)
        check(load().latentmoe_lbl_stats(self.handle, ps.data_ptr(), cn.data_ptr(),
                                         _stream(stream)), "latentmoe_lbl_stats")
        return ps, cn

    def _rows(self, t, name: str, T: int):
        """Row stride of a [T, E] fp32 tensor whose columns are contiguous and whose
        rows do not overlap (a stride of 0, an expanded row, means E to the library)."""
        import torch
        E = self.dims.num_experts
        ld = t.stride(0) if T > 1 and t.dim() == 2 else E
        if not (t.dtype is torch.float32 and t.is_cuda and t.shape == (T, E) and
                (E == 1 or t.stride(1) == 1) and ld >= E):
            raise ValueError(f"{name} must be a float32 CUDA tensor [{T}, {E}] with contiguous "
                             "rows that do not overlap")
        return ld

    def _per_slot(self, t, name: str, T: int, dtype) -> None:
        if not (t.dtype is dtype and t.is_cuda and t.shape == (T, self.k) and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor [{T}, {self.k}]")

    def _sequences(self, T: int, seq_len: int) -> int:
        L = seq_len or T
        _need(L > 0 and T > 0 and T % L == 0, "seq_len must divide the number of tokens")
        return T // L

    def _valid(self, valid, T: int):
        import torch
        if valid is None:
            return None
        _need(valid.is_cuda and valid.dtype in (torch.uint8, torch.bool) and valid.numel() == T and
              valid.is_contiguous(), f"valid must be a contiguous uint8 or bool CUDA tensor [{T}]")
        return valid.data_ptr()

    def balance_loss(self, logits, idx, valid=None, seq_len: int = 0, balance_coef: float = 1.0,
                     z_coef: float = 0.0, stream=None):
        """The router's balance loss of logits [T, E] fp32 and choices idx
        [T, k] int32: {"loss": [total, balance, z], "counts" [S, E] int32,
        "prob_sum" [S, E], "z_sum" [S], "tokens" [S] int32} over S = T /
        seq_len sequences (0: one)."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.balance_loss, logits, idx, valid, seq_len,
                              balance_coef, z_coef)
        T, E = logits.shape[0], self.dims.num_experts
        ld = self._rows(logits, "logits", T)
        self._per_slot(idx, "idx", T, torch.int32)
        S = self._sequences(T, seq_len)
        # new_empty of the inputs: the cheapest way to five small outputs
        loss, prob, z = logits.new_empty(3), logits.new_empty((S, E)), logits.new_empty(S)
        counts, tokens = idx.new_empty((S, E)), idx.new_empty(S)
        st = latentmoe_balance_stats(counts.data_ptr(), prob.data_ptr(), z.data_ptr(),
                                     tokens.data_ptr())
        check(load().latentmoe_balance_loss(
            self.handle, logits.data_ptr(), ld, idx.data_ptr(), self._valid(valid, T), T, seq_len,
            balance_coef, z_coef, ctypes.byref(st), loss.data_ptr(), _stream(None)),
            "latentmoe_balance_loss", self.handle)
        return {"loss": loss, "counts": counts, "prob_sum": prob, "z_sum": z, "tokens": tokens}

    def balance_loss_from_stats(self, stats, balance_coef: float = 1.0, z_coef: float = 0.0,
                                stream=None):
        """loss [3] from (summed) stats as returned by balance_loss."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.balance_loss_from_stats, stats, balance_coef, z_coef)
        c = stats["counts"]
        S, E = c.shape[0], self.dims.num_experts
        for name, shape, dt in (("counts", (S, E), torch.int32), ("prob_sum", (S, E), torch.float32),
                                ("z_sum", (S,), torch.float32), ("tokens", (S,), torch.int32)):
            t = stats[name]
            _need(t.is_cuda and t.dtype == dt and tuple(t.shape) == shape and t.is_contiguous(),
                  f"{name} must be a contiguous {dt} CUDA tensor {list(shape)}")
        loss = torch.empty((3,), dtype=torch.float32, device=c.device)
        st = latentmoe_balance_stats(*(stats[n].data_ptr() for n in
                                       ("counts", "prob_sum", "z_sum", "tokens")))
        check(load().latentmoe_balance_loss_from_stats(self.handle, ctypes.byref(st), S,
                                                       balance_coef, z_coef, loss.data_ptr(),
                                                       _stream(None)),
              "latentmoe_balance_loss_from_stats", self.handle)
        return loss

    def router_backward(self, logits, idx, counts, tokens, d_gates=None, valid=None,
                        seq_len: int = 0, balance_coef: float = 1.0, z_coef: float = 0.0,
                        d_loss=None, out=None, stream=None):
        """d logits [T, E] fp32 of d_loss * loss[0] + sum d_gates * gates."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.router_backward, logits, idx, counts, tokens, d_gates,
                              valid, seq_len, balance_coef, z_coef, d_loss, out)
        T, E = logits.shape[0], self.dims.num_experts
        ld = self._rows(logits, "logits", T)
        S = self._sequences(T, seq_len)
        if idx is not None:
            self._per_slot(idx, "idx", T, torch.int32)
        if d_gates is not None:
            self._per_slot(d_gates, "d_gates", T, torch.float32)
        for t, name, shape in ((counts, "counts", (S, E)), (tokens, "tokens", (S,))):
            if not (t.dtype is torch.int32 and t.is_cuda and t.shape == shape and
                    t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {list(shape)}")
        if d_loss is not None:
            _need(d_loss.is_cuda and d_loss.dtype == torch.float32 and d_loss.numel() == 1,
                  "d_loss must be one float32 on the GPU")
        if out is None:
            out = logits.new_empty((T, E))
        check(load().latentmoe_router_backward(
            self.handle, logits.data_ptr(), ld, _ptr(idx), _ptr(d_gates), self._valid(valid, T),
            counts.data_ptr(), tokens.data_ptr(), T, seq_len, balance_coef, z_coef, _ptr(d_loss),
            out.data_ptr(), self._rows(out, "out", T), _stream(None)),
            "latentmoe_router_backward", self.handle)
        return out

    def status(self) -> int:
        v = ctypes.c_uint32(0)
        load().latentmoe_get_status(self.handle, ctypes.byref(v))
        return v.value

    def set_profiling(self, slots: int) -> None:
        check(load().latentmoe_set_profiling(self.handle, slots), "latentmoe_set_profiling")

    def stage_times(self, slot: int):
        n = load().latentmoe_num_stages()
        buf = (ctypes.c_float * n)()
        check(load().latentmoe_get_stage_times(self.handle, slot, buf, n),
              "latentmoe_get_stage_times")
        return {stage_name(i): buf[i] for i in range(n)}

    def fp8_state(self):
        """{"scales": [s_z, s_h] for the next forward, "last_amax": the last
        forward's maxima, "steps": forwards entered into the history}."""
        sc = (ctypes.c_float * FP8_TENSORS)()
        am = (ctypes.c_float * FP8_TENSORS)()
        st = _i64(0)
        check(load().latentmoe_get_fp8_state(self.handle, sc, am, ctypes.byref(st)),
              "latentmoe_get_fp8_state")
        return {"scales": list(sc), "last_amax": list(am), "steps": st.value}

    def fp8_codes(self, T: int, device, stream=None):
        """(z codes [T*k, l], h codes [T*k, F]) uint8 of the last forward."""
        import torch
        S = T * self.k
        zc = torch.empty((S, self.dims.latent), dtype=torch.uint8, device=device)
        hc = torch.empty((S, self.dims.ffn), dtype=torch.uint8, device=device)
        check(load().latentmoe_get_fp8_codes(self.handle, zc.data_ptr(), hc.data_ptr(),
                                             _stream(stream)), "latentmoe_get_fp8_codes")
        return zc, hc

    def set_fp8_scales(self, scales) -> None:
        """Scales for z, h[, x, c, shared hidden]; the ones not given are 1."""
        vals = list(scales) + [1.0] * (FP8_TENSORS - len(scales))
        sc = (ctypes.c_float * FP8_TENSORS)(*vals)
        check(load().latentmoe_set_fp8_scales(self.handle, sc), "latentmoe_set_fp8_scales")

    def fp8_weight_scales(self):
        """[3, E] list of lists: scales of W_g, W_u, W_d per expert."""
        return self.fp8_all_weight_scales()[0]

    def fp8_all_weight_scales(self):
        """([3, E] expert scales, {w_dn, w_up, w_gs, w_us, w_ds} dense scales)."""
        E = self.dims.num_experts
        buf = (ctypes.c_float * (3 * E + 5))()
        check(load().latentmoe_get_fp8_weight_scales(self.handle, buf),
              "latentmoe_get_fp8_weight_scales")
        dense = dict(zip(("w_dn", "w_up", "w_gs", "w_us", "w_ds"), buf[3 * E:3 * E + 5]))
        return [list(buf[m * E:(m + 1) * E]) for m in range(3)], dense

    def fp8_dense_codes(self, T: int, device, stream=None):
        """(x codes [T, d], c codes [T, l], shared hidden codes [T, F_s] or None)."""
        import torch
        xc = torch.empty((T, self.dims.hidden), dtype=torch.uint8, device=device)
        cc = torch.empty((T, self.dims.latent), dtype=torch.uint8, device=device)
        sc = torch.empty((T, self.dims.shared_ffn), dtype=torch.uint8, device=device) \
            if self.dims.shared_ffn else None
        check(load().latentmoe_get_fp8_dense_codes(self.handle, xc.data_ptr(), cc.data_ptr(),
                                                   _ptr(sc), _stream(stream)),
              "latentmoe_get_fp8_dense_codes")
        return xc, cc, sc

    def set_capacity(self, capacity: int, group_size: int = 1, max_rounds: int = 0) -> None:
        """Multi-round fixed-capacity expert schedule (capacity 0: one pass)."""
        check(load().latentmoe_set_capacity(self.handle, capacity, group_size, max_rounds),
              "latentmoe_set_capacity", self.handle)

    def rounds(self, device="cuda"):
        """{"needed", "left_over", "launched", "take" [launched, E] int32} of the last forward."""
        import torch
        info = (ctypes.c_int32 * 3)()
        check(load().latentmoe_get_rounds(self.handle, None, info), "latentmoe_get_rounds")
        take = torch.empty((info[2], self.dims.num_experts), dtype=torch.int32, device=device)
        check(load().latentmoe_get_rounds(self.handle, take.data_ptr(), info),
              "latentmoe_get_rounds")
        return {"needed": info[0], "left_over": info[1], "launched": info[2], "take": take}

    def set_sm_pairs(self, enable: bool) -> None:
        check(load().latentmoe_set_sm_pairs(self.handle, int(enable)),
              "latentmoe_set_sm_pairs")

    def set_expert_fusion(self, mode) -> None:
        """0 (or False): two expert launches; 1 (or True): one fused launch where
        the shapes allow; 2: automatic (the default)."""
        check(load().latentmoe_set_expert_fusion(self.handle, int(mode)),
              "latentmoe_set_expert_fusion", self.handle)

    def set_pdl(self, enable: bool) -> None:
        check(load().latentmoe_set_pdl(self.handle, 1 if enable else 0), "latentmoe_set_pdl",
              self.handle)

    def launch_count(self) -> int:
        v = _i64(0)
        check(load().latentmoe_get_launch_count(self.handle, ctypes.byref(v)),
              "latentmoe_get_launch_count")
        return v.value


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _dtype_code(t, name: str) -> int:
    import torch
    _need(t.dtype in (torch.bfloat16, torch.float32), f"{name} must be bfloat16 or float32")
    return FP32 if t.dtype == torch.float32 else BF16


class Muon:
    """A handle that orthogonalises updates of a stack of ``batch`` matrices
    [rows, cols] by Newton-Schulz products. ``coefs``: one (a, b, c) for every
    step, or a list of ``steps`` of them; None for the library's default."""

    def __init__(self, rows: int, cols: int, batch: int = 1, steps: int = 5, coefs=None,
                 eps: float = 1e-7):
        lib = load()
        arr = None
        if coefs is not None:
            flat = [float(v) for c in coefs for v in (c if hasattr(c, "__len__") else (c,))]
            if len(flat) == 3:
                flat = flat * steps
            _need(len(flat) == 3 * steps, "coefs must be (a, b, c) or one (a, b, c) per step")
            arr = (ctypes.c_float * len(flat))(*flat)
        self.dims = latentmoe_muon_dims(batch, rows, cols, steps,
                                        ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
                                        if arr is not None else None, eps)
        h = _c_void_p()
        check(lib.latentmoe_muon_create(ctypes.byref(self.dims), ctypes.byref(h)),
              "latentmoe_muon_create")
        self.dims.coefs = None  # the library has copied them
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            load().latentmoe_muon_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, code: int, what: str) -> None:
        if code != OK:
            raise LatentMoEError(code, what, load().latentmoe_muon_last_cuda_error(self.handle))

    def _matrices(self, t, name: str) -> None:
        d = self.dims
        _need(t.is_cuda and t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
        shape = tuple(t.shape) if t.dim() == 3 else (1,) + tuple(t.shape)
        _need(shape == (d.batch, d.rows, d.cols),
              f"{name} must be [{d.batch}, {d.rows}, {d.cols}], got {list(t.shape)}")

    def orthogonalize(self, g, out=None, stream=None):
        """The orthogonalised g (bf16 or fp32), in bf16."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.orthogonalize, g, out)
        self._matrices(g, "g")
        if out is None:
            out = torch.empty_like(g, dtype=torch.bfloat16)
        else:
            self._matrices(out, "out")
            _need(out.dtype == torch.bfloat16, "out must be bfloat16")
        self._check(load().latentmoe_muon_orthogonalize(
            self.handle, g.data_ptr(), _dtype_code(g, "g"), out.data_ptr(), _stream(None)),
            "latentmoe_muon_orthogonalize")
        return out

    def step(self, w, g, momentum, lr: float, momentum_coef: float = 0.95,
             weight_decay: float = 0.0, scale: float = 1.0, nesterov: bool = True,
             stream=None) -> None:
        """One optimiser step: momentum (fp32) and w (bf16 or fp32) in place."""
        import torch
        for t, name in ((w, "w"), (g, "g"), (momentum, "momentum")):
            self._matrices(t, name)
        _need(momentum.dtype == torch.float32, "momentum must be float32")
        u = latentmoe_muon_update(g.data_ptr(), momentum.data_ptr(), w.data_ptr(),
                                  _dtype_code(g, "g"), _dtype_code(w, "w"), int(nesterov), lr,
                                  momentum_coef, weight_decay, scale)
        self._check(load().latentmoe_muon_step(self.handle, ctypes.byref(u), _stream(stream)),
                    "latentmoe_muon_step")

    def set_sm_pairs(self, mode: int) -> None:
        """0: 128 x 128 tiles on single SMs; 1: 256 x 256 on SM pairs; 3: 128 x 64
        on single SMs; 2: automatic."""
        self._check(load().latentmoe_muon_set_sm_pairs(self.handle, int(mode)),
                    "latentmoe_muon_set_sm_pairs")

    def status(self) -> int:
        v = ctypes.c_uint32(0)
        load().latentmoe_muon_get_status(self.handle, ctypes.byref(v))
        return v.value

    def launch_count(self) -> int:
        v = _i64(0)
        self._check(load().latentmoe_muon_get_launch_count(self.handle, ctypes.byref(v)),
                    "latentmoe_muon_get_launch_count")
        return v.value


_raw_device = None  # () -> ordinal of the current device


def _device() -> int:
    global _raw_device
    if _raw_device is None:
        import torch
        torch.cuda.current_device()  # CUDA is initialised from here on
        _raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _raw_device()


# Checks of the block's operators. A small call is half Python, so the current device is
# asked for once a call, and a message is put together only where it is raised.
# get_device is -1 for a host tensor; device pointers are the current device's.
def _not_here(t, name: str, dev: int) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")


def _token_rows(t, name: str, T: int, d: int, dtypes, dev: int) -> int:
    """Row stride of a [T, d] tensor whose rows are contiguous and do not overlap."""
    if t.get_device() != dev or t.dtype not in dtypes or t.shape != (T, d):
        _not_here(t, name, dev)
        raise ValueError(f"{name} must be [{T}, {d}] of type "
                         f"{' or '.join(str(x) for x in dtypes)}, got {list(t.shape)} {t.dtype}")
    step, inner = t.stride()
    ld = step if T > 1 else d
    if (inner != 1 and d > 1) or ld < d:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return ld


def _matrix(t, name: str, rows: int, cols: int, dtype, dev: int) -> int:
    """Address of a contiguous [rows, cols]."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != (rows, cols) or \
            not t.is_contiguous():
        _not_here(t, name, dev)
        raise ValueError(f"{name} must be a contiguous {dtype} [{rows}, {cols}], got "
                         f"{list(t.shape)} {t.dtype}")
    return t.data_ptr()


class GatedFFN:
    """A handle on a gated feed-forward block y = (SiLU(x w_g^T) * (x w_u^T)) w_d^T of
    width ``d`` and hidden width ``F`` (multiples of 8) for up to ``max_tokens`` rows;
    ``training``: with the gradient's workspace. Weights are the caller's, bf16, and
    passed at every call: w_g, w_u [F, d], w_d [d, F]."""

    def __init__(self, d: int, F: int, max_tokens: int = 1, training: bool = False):
        self.dims = latentmoe_ffn_dims(d, F, max_tokens, int(training))
        self.d, self.F, self.device = d, F, None
        h = _c_void_p()
        check(load().latentmoe_ffn_create(ctypes.byref(self.dims), ctypes.byref(h)),
              "latentmoe_ffn_create")
        self.handle = h
        self.device = _device()

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            load().latentmoe_ffn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, code: int, what: str) -> None:
        if code != OK:
            raise LatentMoEError(code, what, load().latentmoe_ffn_last_cuda_error(self.handle))

    def _weights(self, w_g, w_u, w_d, b16, dev: int):
        d, F = self.d, self.F
        if dev != self.device:
            raise ValueError("the handle belongs to another device than the current one")
        return latentmoe_ffn_weights(_matrix(w_g, "w_g", F, d, b16, dev),
                                     _matrix(w_u, "w_u", F, d, b16, dev),
                                     _matrix(w_d, "w_d", d, F, b16, dev))

    def forward(self, x, w_g, w_u, w_d, save: bool = False, out=None, stream=None):
        """y [T, d] bf16 of x [T, d] bf16 (rows may be strided); with ``save`` (y, gate,
        up), the latter [T, F] bf16 for ``backward``."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.forward, x, w_g, w_u, w_d, save, out)
        if x.dim() != 2:
            raise ValueError("x must be [T, d]")
        T, d, F, b16, cur, dev = x.shape[0], self.d, self.F, torch.bfloat16, _device(), x.device
        ld_x, ld_y = _token_rows(x, "x", T, d, (b16,), cur), d
        w = self._weights(w_g, w_u, w_d, b16, cur)
        if out is None:
            y = torch.empty((T, d), dtype=b16, device=dev)
        else:
            y, ld_y = out, _token_rows(out, "out", T, d, (b16,), cur)
        gate = up = at_gate = at_up = None
        if save:
            gate = torch.empty((T, F), dtype=b16, device=dev)
            up = torch.empty((T, F), dtype=b16, device=dev)
            at_gate, at_up = gate.data_ptr(), up.data_ptr()
        code = load().latentmoe_ffn_forward(self.handle, ctypes.byref(w), x.data_ptr(), ld_x,
                                            y.data_ptr(), ld_y, at_gate, at_up, T, _stream(None))
        if code != OK:
            self._check(code, "latentmoe_ffn_forward")
        return (y, gate, up) if save else y

    def backward(self, dy, x, gate, up, w_g, w_u, w_d, dw_dtype=None, out=None,
                 accumulate: bool = False, need=("dx", "dw_g", "dw_u", "dw_d"), stream=None):
        """{"dx" [T, d] bf16, "dw_g", "dw_u" [F, d], "dw_d" [d, F]} of dy [T, d]; the
        weights' gradients are bf16, or dw_dtype=torch.float32. ``out``: a dict of tensors
        to write to (their type counts), added to with ``accumulate`` (fp32 weights'
        gradients). ``need``: the ones that are wanted."""
        import torch
        if stream is not None:
            return _on_stream(stream, self.backward, dy, x, gate, up, w_g, w_u, w_d, dw_dtype, out,
                              accumulate, need)
        if dy.dim() != 2:
            raise ValueError("dy must be [T, d]")
        T, d, F, b16, cur, dev = dy.shape[0], self.d, self.F, torch.bfloat16, _device(), dy.device
        ld_dy, ld_x = _token_rows(dy, "dy", T, d, (b16,), cur), _token_rows(x, "x", T, d, (b16,), cur)
        w = self._weights(w_g, w_u, w_d, b16, cur)
        out = out or {}
        dt = dw_dtype or next((out[n].dtype for n in ("dw_g", "dw_u", "dw_d")
                               if n in need and n in out), b16)
        got, at, ld_dx = {}, [None] * 4, 0
        for i, (n, rows, cols) in enumerate((("dx", T, d), ("dw_g", F, d), ("dw_u", F, d),
                                             ("dw_d", d, F))):
            if n not in need:
                continue
            if n not in out:
                if accumulate and i:
                    raise ValueError("accumulate needs the weights' gradients in out")
                t = torch.empty((rows, cols), dtype=dt if i else b16, device=dev)
                at[i] = t.data_ptr()
            elif i:
                t = out[n]
                at[i] = _matrix(t, n, rows, cols, dt, cur)
            else:
                t = out[n]
                at[i], ld_dx = t.data_ptr(), _token_rows(t, n, T, d, (b16,), cur)
            got[n] = t
        if dt is not b16 and dt is not torch.float32:
            raise ValueError("the weights' gradients must be bfloat16 or float32")
        g = latentmoe_ffn_grad(dy.data_ptr(), x.data_ptr(), _matrix(gate, "gate", T, F, b16, cur),
                               _matrix(up, "up", T, F, b16, cur), at[0], at[1], at[2], at[3], ld_dy,
                               ld_x, ld_dx, BF16 if dt is b16 else FP32, 1 if accumulate else 0)
        code = load().latentmoe_ffn_backward(self.handle, ctypes.byref(w), ctypes.byref(g), T,
                                             _stream(None))
        if code != OK:
            self._check(code, "latentmoe_ffn_backward")
        return got

    def set_sm_pairs(self, mode: int) -> None:
        """0: 128 x 128 tiles on single SMs; 1: 256 x 256 on SM pairs; 2: automatic;
        3: the kernel for few tokens."""
        self._check(load().latentmoe_ffn_set_sm_pairs(self.handle, int(mode)),
                    "latentmoe_ffn_set_sm_pairs")

    def status(self) -> int:
        v = ctypes.c_uint32(0)
        load().latentmoe_ffn_get_status(self.handle, ctypes.byref(v))
        return v.value

    def launch_count(self) -> int:
        v = _i64(0)
        self._check(load().latentmoe_ffn_get_launch_count(self.handle, ctypes.byref(v)),
                    "latentmoe_ffn_get_launch_count")
        return v.value


def _norm_weight(weight, d: int, dev: int) -> int:
    if weight.get_device() != dev or weight.shape != (d,) or not weight.is_contiguous():
        _not_here(weight, "weight", dev)
        raise ValueError(f"weight must be a contiguous [{d}]")
    return _dtype_code(weight, "weight")


SCALE_BLOCK = 128  # channels of an E4M3 scale block


def rms_norm(x, weight, eps: float = 1e-6, residual=None, quantize: Optional[str] = None,
             keep_y: bool = False, y_dtype=None, out_sum=None, stream=None):
    """RMS norm of s = x + residual, rows x [T, d] (bf16 or fp32), weight [d]:
    {"y": [T, d], "rstd": [T] fp32 for rms_norm_backward, "sum": s in the residual's
    type where one is given}. quantize "token" or "block": y as E4M3 "codes" (uint8
    [T, d]) with "scales" fp32 [T, 1] or [T, ceil(d / 128)] instead of y, or beside
    it with keep_y. y has x's type unless y_dtype says otherwise. out_sum: where s
    goes, e.g. the residual itself."""
    import torch
    if stream is not None:
        return _on_stream(stream, rms_norm, x, weight, eps, residual, quantize, keep_y, y_dtype,
                          out_sum)
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    if quantize not in (None, "token", "block"):
        raise ValueError('quantize must be None, "token" or "block"')
    # torch.empty, not new_empty: half the time of a call that takes 3 us
    f32, empty, dev, dt, cur = torch.float32, torch.empty, x.device, x.dtype, _device()
    both = (torch.bfloat16, f32)
    T, d = x.shape
    ld_x, w_code = _token_rows(x, "x", T, d, both, cur), _norm_weight(weight, d, cur)
    rstd = empty(T, dtype=f32, device=dev)
    out = {"rstd": rstd}
    r = s = y = codes = scales = None
    ld_r = ld_s = r_code = y_code = block = 0
    if residual is not None:
        ld_r, r_dt = _token_rows(residual, "residual", T, d, both, cur), residual.dtype
        r = residual.data_ptr()
        r_code = FP32 if r_dt is f32 else BF16
        if out_sum is None:
            s_out, ld_s = empty((T, d), dtype=r_dt, device=dev), d
        else:
            s_out, ld_s = out_sum, _token_rows(out_sum, "out_sum", T, d, (r_dt,), cur)
        out["sum"] = s_out
        s = s_out.data_ptr()
    elif out_sum is not None:
        raise ValueError("out_sum needs a residual")
    if quantize is None or keep_y:
        out["y"] = y_out = empty((T, d), dtype=y_dtype or dt, device=dev)
        y, y_code = y_out.data_ptr(), _dtype_code(y_out, "y")
    if quantize is not None:
        n = 1
        if quantize == "block":
            block, n = SCALE_BLOCK, -(-d // SCALE_BLOCK)
        out["codes"] = empty((T, d), dtype=torch.uint8, device=dev)
        out["scales"] = empty((T, n), dtype=f32, device=dev)
        codes, scales = out["codes"].data_ptr(), out["scales"].data_ptr()
    a = latentmoe_norm(x.data_ptr(), r, weight.data_ptr(), s, y, codes, scales, rstd.data_ptr(),
                       ld_x, ld_r, ld_s, d, d, FP32 if dt is f32 else BF16, r_code, w_code,
                       y_code, block, eps)
    code = load().latentmoe_rms_norm(ctypes.byref(a), T, d, _stream(None))
    if code != OK:
        check(code, "latentmoe_rms_norm")
    return out


def rms_norm_backward(dy, s, weight, rstd, d_sum=None, dw: bool = True, dx_bf16: bool = False,
                      stream=None):
    """Gradient of rms_norm: {"dx": [T, d] of s's type, the gradient of x and of the
    residual alike, "dw": [d] fp32}. s: the norm's "sum" (its x where there was no
    residual); d_sum: the gradient that reached it from further down the stream.
    dx_bf16 (fp32 streams): "dx16" as well, dx in bf16."""
    import torch
    if stream is not None:
        return _on_stream(stream, rms_norm_backward, dy, s, weight, rstd, d_sum, dw, dx_bf16)
    if dy.dim() != 2:
        raise ValueError("dy must be [T, d]")
    f32, empty, dev, cur = torch.float32, torch.empty, dy.device, _device()
    both = (torch.bfloat16, f32)
    T, d = dy.shape
    if rstd.get_device() != cur or rstd.dtype is not f32 or rstd.shape != (T,) or \
            not rstd.is_contiguous():
        _not_here(rstd, "rstd", cur)
        raise ValueError(f"rstd must be a contiguous float32 [{T}]")
    ld_dy, ld_s = _token_rows(dy, "dy", T, d, both, cur), _token_rows(s, "s", T, d, both, cur)
    w_code = _norm_weight(weight, d, cur)
    ld_ds = 0 if d_sum is None else _token_rows(d_sum, "d_sum", T, d, (s.dtype,), cur)
    dx = empty((T, d), dtype=s.dtype, device=dev)
    out = {"dx": dx}
    dx16 = ws = grad = None
    size = 0
    if dx_bf16:
        if s.dtype is not f32:
            raise ValueError("dx_bf16 is for float32 streams")
        out["dx16"] = empty((T, d), dtype=torch.bfloat16, device=dev)
        dx16 = out["dx16"].data_ptr()
    lib = load()
    if dw:
        size = lib.latentmoe_rms_norm_backward_workspace(T, d)
        ws = empty(size, dtype=torch.uint8, device=dev)
        out["dw"] = empty(d, dtype=f32, device=dev)
        grad = out["dw"].data_ptr()
    a = latentmoe_norm_grad(dy.data_ptr(), s.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                            _ptr(d_sum), dx.data_ptr(), dx16, grad, ld_dy, ld_s, ld_ds, d, d,
                            FP32 if dy.dtype is f32 else BF16, FP32 if s.dtype is f32 else BF16,
                            w_code)
    code = lib.latentmoe_rms_norm_backward(ctypes.byref(a), T, d, _ptr(ws), size, _stream(None))
    if code != OK:
        check(code, "latentmoe_rms_norm_backward")
    return out


def _gradient_table(grads, out):
    import array
    import torch
    grads = list(grads)
    _need(len(grads) > 0, "no gradients")
    _need(out is None or len(out) == len(grads), "out must have one tensor for each gradient")
    bf16, f32, dev = torch.bfloat16, torch.float32, _device()
    flat = array.array("q")
    push = flat.extend
    for i, g in enumerate(grads):
        dt, n = g.dtype, g.numel()
        # get_device is -1 for a host tensor
        if not ((dt is bf16 or dt is f32) and g.get_device() == dev and g.is_contiguous()):
            raise ValueError("gradients must be contiguous bfloat16 or float32 tensors on the "
                             "current CUDA device")
        at = to = g.data_ptr()
        if out is not None:
            o = out[i]
            if not (o.dtype is dt and o.get_device() == dev and o.is_contiguous() and
                    o.numel() == n):
                raise ValueError("out must have the gradients' sizes, types and device, and be "
                                 "contiguous")
            to = o.data_ptr()
        push((at, to, n, FP32 if dt is f32 else BF16))
    lib = load()
    ws = torch.empty(lib.latentmoe_grad_workspace(len(grads)), dtype=torch.uint8,
                     device=grads[0].device)
    norm = torch.empty(1, dtype=f32, device=grads[0].device)
    return flat, len(grads), norm, ws


def gradient_norm(grads, stream=None):
    """sqrt of the sum of all squares of the tensors (bf16 or fp32), as fp32 [1]."""
    if stream is not None:
        return _on_stream(stream, gradient_norm, grads)
    flat, n, norm, ws = _gradient_table(grads, None)
    check(load().latentmoe_grad_norm(flat.buffer_info()[0], n, norm.data_ptr(), ws.data_ptr(),
                                     ws.numel(), _stream(None)), "latentmoe_grad_norm")
    return norm


def clip_gradients(grads, max_norm: float, eps: float = 1e-6, out=None, stream=None):
    """Scales the tensors by min(1, max_norm / (norm + eps)) in place, or into the
    tensors of ``out``; returns the norm before it, fp32 [1]."""
    if stream is not None:
        return _on_stream(stream, clip_gradients, grads, max_norm, eps, out)
    flat, n, norm, ws = _gradient_table(grads, out)
    check(load().latentmoe_grad_clip(flat.buffer_info()[0], n, max_norm, eps, norm.data_ptr(),
                                     ws.data_ptr(), ws.numel(), _stream(None)),
          "latentmoe_grad_clip")
    return norm


def stage_name(i: int) -> str:
    return load().latentmoe_stage_name(i).decode()


def debug_gemm(A, B, C, M: int, N: int, K: int, mode: int, stream=None) -> int:
    return load().latentmoe_debug_gemm(A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N, K, mode,
                                       _stream(stream))


def debug_grouped_gemm(A, B, C, offsets, groups: int, M: int, N: int, K: int, mode: int,
                       stream=None) -> int:
    return load().latentmoe_debug_grouped_gemm(A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                               offsets.data_ptr(), groups, M, N, K, mode,
                                               _stream(stream))


def quantize_e4m3(src, codes, scales, stream=None) -> int:
    """src bf16 [G, R, C] (device) -> codes uint8 [G, R, C], scales fp32 [G]."""
    G, R, C = src.shape
    return load().latentmoe_quantize_e4m3(src.data_ptr(), G, R, C, codes.data_ptr(),
                                          scales.data_ptr(), _stream(stream))


def debug_grouped_gemm_e4m3(A, B, scales, C, amax, offsets, groups: int, M: int, N: int, K: int,
                            mode: int, stream=None) -> int:
    return load().latentmoe_debug_grouped_gemm_e4m3(
        A.data_ptr(), B.data_ptr(), scales.data_ptr(), C.data_ptr(), _ptr(amax),
        offsets.data_ptr(), groups, M, N, K, mode, _stream(stream))


def debug_status() -> int:
    v = ctypes.c_uint32(0)
    load().latentmoe_debug_status(ctypes.byref(v))
    return v.value
