"""Python binding of the gsfp8 C ABI (``include/gsfp8.h``).

Argument marshalling only: every function takes torch tensors (device
memory) and the current CUDA stream, passes raw pointers and sizes to the
same-named C entry point of ``libgsfp8.so`` and raises ``GsError`` on a
non-zero status.  There is no fallback: if the shared library is missing,
importing this package raises ``ImportError``.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

__all__ = [
    "GS_OK", "GS_F16", "GS_BF16", "GS_F32", "GS_E4M3", "GS_E5M2", "GsError", "TensorList",
    "gs_status_str", "gs_version", "gs_tensor_list_create", "gs_unscale_check_update",
    "gs_scaler_state_get", "gs_scaler_state_set", "fp8_quant_block", "fp8_quant_tensor",
    "fp8_dequant", "gs_ws_bytes", "gs_device_status", "lib_path",
    "gs_unscale_check_update_noalloc", "gs_noalloc_limits", "fp8_quant_mx", "fp8_dequant_mx",
    "gs_unscale_check_update_hysteresis", "fp8_quant_tensor_delayed",
    "gs_unscale_check_update_norm", "ParamList", "gs_param_list_create", "gs_master_update_sgd",
    "AdamWList", "gs_adamw_list_create", "gs_master_update_adamw", "gs_layernorm_fwd",
    "gs_layernorm_bwd", "gs_layernorm_ws_bytes", "gs_token_logprob", "gs_token_logprob_bwd",
    "GS_MAX_TOP", "GS_MOMENTS_F32", "GS_MOMENTS_E4M3", "GS_MXFP4", "GS_NVFP4", "fp4_scale_bytes",
    "fp4_quant", "fp4_dequant", "fp4_gemm_block_scaled", "gs_policy_loss", "gs_policy_loss_ws_bytes",
    "MuonList", "gs_muon_list_create", "gs_master_update_muon",
]

GS_OK, GS_ERR_NULL, GS_ERR_SHAPE, GS_ERR_DTYPE, GS_ERR_ARG, GS_ERR_CUDA, GS_ERR_TIMEOUT = range(7)
GS_F16, GS_BF16, GS_F32 = 0, 1, 2
GS_E4M3, GS_E5M2 = 0, 1
GS_MOMENTS_F32, GS_MOMENTS_E4M3 = 0, 1
GS_MAX_TOP = 32
GS_MXFP4, GS_NVFP4 = 0, 1
GS_LOSS_TOKEN_MEAN, GS_LOSS_SEQUENCE_MEAN, GS_LOSS_SUM = 0, 1, 2

_DTYPES = {torch.float16: GS_F16, torch.bfloat16: GS_BF16, torch.float32: GS_F32}
_FMTS4 = {"mxfp4": GS_MXFP4, "nvfp4": GS_NVFP4, GS_MXFP4: GS_MXFP4, GS_NVFP4: GS_NVFP4}
_MUON_SCALES = {"rms": 0, "aspect": 1}
_REDUCTIONS = {"token": GS_LOSS_TOKEN_MEAN, "sequence": GS_LOSS_SEQUENCE_MEAN, "sum": GS_LOSS_SUM}
_FMTS = {"e4m3": GS_E4M3, "e5m2": GS_E5M2, GS_E4M3: GS_E4M3, GS_E5M2: GS_E5M2}


def lib_path() -> str:
    return _build.LIB


def _load_lib() -> ctypes.CDLL:
    if not _build.up_to_date():
        if os.environ.get("GSFP8_BUILD_ON_IMPORT", "1") == "1":
            _build.build()
        elif not os.path.exists(_build.LIB):
            raise ImportError(f"libgsfp8.so not built ({_build.LIB}); run __graft_entry__.build()")
    lib = ctypes.CDLL(_build.LIB)
    i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    ci = ctypes.c_int
    sigs = {
        "gs_status_str": (ctypes.c_char_p, [ci]),
        "gs_last_cuda_error": (ci, []),
        "gs_version": (ctypes.c_char_p, []),
        "gs_tensor_list_create": (ci, [vp, vp, vp, i32, ctypes.POINTER(vp)]),
        "gs_tensor_list_destroy": (ci, [vp]),
        "gs_tensor_list_info": (ci, [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "gs_unscale_check_update": (ci, [vp, vp, vp, vp, vp, f32, f32, i32, vp]),
        "gs_scaler_state_get": (ci, [vp, vp, ctypes.POINTER(f32), ctypes.POINTER(i32), vp]),
        "gs_scaler_state_set": (ci, [vp, vp, f32, i32, vp]),
        "fp8_quant_block": (ci, [vp, ci, i64, i64, i32, i32, ci, vp, vp, vp]),
        "gs_ws_bytes": (ctypes.c_size_t, []),
        "fp8_quant_tensor": (ci, [vp, ci, i64, ci, vp, vp, vp, vp]),
        "fp8_dequant": (ci, [vp, vp, i64, i64, i32, i32, ci, ci, vp, vp]),
        "gs_device_status": (ci, [ctypes.POINTER(i32), vp]),
        "gs_unscale_check_update_norm": (ci, [vp, vp, vp, vp, vp, f32, f32, i32, vp, vp]),
        "gs_param_list_create": (ci, [vp, vp, vp, vp, i32, ctypes.POINTER(vp)]),
        "gs_param_list_destroy": (ci, [vp]),
        "gs_master_update_sgd": (ci, [vp, f32, f32, vp, vp, vp]),
        "gs_unscale_check_update_hysteresis": (ci, [vp, vp, vp, vp, vp, vp, f32, f32, i32, i32, i32,
                                                    f32, vp]),
        "fp8_quant_tensor_delayed": (ci, [vp, ci, i64, ci, vp, vp, i32, vp, vp, vp, vp]),
        "fp8_quant_mx": (ci, [vp, ci, i64, i64, ci, vp, vp, vp]),
        "fp8_dequant_mx": (ci, [vp, vp, i64, i64, ci, ci, vp, vp]),
        "gs_unscale_check_update_noalloc": (ci, [vp, vp, vp, i32, vp, vp, vp, vp, f32, f32, i32, vp]),
        "gs_noalloc_limits": (ci, [ctypes.POINTER(i32), ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "fp8_gemm_block_scaled": (ci, [vp, vp, vp, vp, i64, i64, i64, ci, ci, ci, vp, vp]),
        "gs_test_set_stall": (ci, [ci]),
        "gs_test_adamw_root": (ci, [vp, vp, i64, vp]),
        "gs_layernorm_fwd": (ci, [vp, i64, ci, i64, i64, vp, vp, ci, f32, vp, i64, vp, vp, vp]),
        "gs_layernorm_ws_bytes": (ctypes.c_size_t, [i64, i64]),
        "gs_layernorm_bwd": (ci, [vp, i64, vp, i64, ci, i64, i64, vp, ci, vp, vp, vp, i64, vp, vp,
                                  ci, vp, vp]),
        "gs_token_logprob": (ci, [vp, i64, ci, i64, i64, vp, vp, vp, vp, i32, vp, vp, vp]),
        "gs_token_logprob_bwd": (ci, [vp, i64, ci, i64, i64, vp, vp, vp, vp, vp, vp, vp, i64, ci,
                                      vp]),
        "gs_muon_list_create": (ci, [vp, vp, vp, ci, vp, vp, vp, i32, ctypes.POINTER(vp)]),
        "gs_muon_list_destroy": (ci, [vp]),
        "gs_master_update_muon": (ci, [vp, f32, f32, f32, ci, i32, ci, f32, vp, vp, vp]),
        "fp4_scale_bytes": (ctypes.c_size_t, [i64, i64, ci]),
        "fp4_quant": (ci, [vp, i64, ci, i64, i64, ci, vp, vp, vp, vp, vp, vp, vp]),
        "fp4_dequant": (ci, [vp, vp, vp, i64, i64, ci, ci, vp, i64, vp]),
        "fp4_gemm_block_scaled": (ci, [vp, vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, vp, i64, vp]),
        "gs_policy_loss_ws_bytes": (ctypes.c_size_t, [i64, i64]),
        "gs_policy_loss": (ci, [vp, vp, vp, vp, i64, vp, i64, vp, i64, f32, f32, f32, f32, ci, vp, vp,
                                vp, vp, vp, vp]),
        "gs_adamw_list_create": (ci, [vp, vp, vp, ci, ci, vp, vp, vp, vp, vp, vp, i32,
                                      ctypes.POINTER(vp)]),
        "gs_adamw_list_destroy": (ci, [vp]),
        "gs_master_update_adamw": (ci, [vp, f32, f32, f32, f32, f32, f32, vp, vp, vp,
                                        ctypes.c_uint32, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load_lib()


class GsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.gs_status_str(status).decode()
        if status == GS_ERR_CUDA:
            msg += f" (cudaError {_lib.gs_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


def _check(status: int, where: str) -> None:
    if status != GS_OK:
        raise GsError(status, where)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


# The current stream's handle without the Stream object around it (3 us of a
# call on a Grace core, more than the launch); None where torch has no CUDA.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_cuda_is_up = torch.cuda.is_initialized
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _cuda_is_up():
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _contig(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gs_status_str(status: int) -> str:
    return _lib.gs_status_str(status).decode()


def gs_version() -> str:
    return _lib.gs_version().decode()


def gs_ws_bytes() -> int:
    return int(_lib.gs_ws_bytes())


class TensorList:
    """Owns a ``gs_tensor_list`` handle (the device chunk table of one
    gradient list).  Keeps references to the tensors it points into."""

    def __init__(self, grads: list[torch.Tensor], outs: list[torch.Tensor]):
        if len(grads) != len(outs):
            raise ValueError("grads and outs differ in length")
        for g, o in zip(grads, outs):
            _contig(g, "grad")
            _contig(o, "out")
            if g.dtype != torch.float16 or o.dtype != torch.float32 or g.numel() != o.numel():
                raise ValueError("each grad must be float16 and its out float32 of equal numel")
        n = len(grads)
        self._keep = (list(grads), list(outs))
        gp = (ctypes.c_void_p * max(n, 1))(*[g.data_ptr() for g in grads])
        op = (ctypes.c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
        ne = (ctypes.c_int64 * max(n, 1))(*[g.numel() for g in grads])
        h = ctypes.c_void_p()
        _check(_lib.gs_tensor_list_create(gp, op, ne, n, ctypes.byref(h)), "gs_tensor_list_create")
        self.handle = h

    def info(self) -> tuple[int, int]:
        total, chunks = ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.gs_tensor_list_info(self.handle, ctypes.byref(total), ctypes.byref(chunks)),
               "gs_tensor_list_info")
        return total.value, chunks.value

    def close(self) -> None:
        if getattr(self, "handle", None):
            _lib.gs_tensor_list_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gs_tensor_list_create(grads: list[torch.Tensor], outs: list[torch.Tensor]) -> TensorList:
    return TensorList(grads, outs)


def gs_unscale_check_update(tlist: TensorList, scale: torch.Tensor, growth_tracker: torch.Tensor,
                            found_inf: torch.Tensor, skipped: torch.Tensor | None = None,
                            growth_factor: float = 2.0, backoff_factor: float = 0.5,
                            growth_interval: int = 2000, stream=None) -> None:
    _check(_lib.gs_unscale_check_update(tlist.handle, _ptr(scale), _ptr(growth_tracker),
                                        _ptr(found_inf), _ptr(skipped), growth_factor,
                                        backoff_factor, growth_interval, _stream(stream)),
           "gs_unscale_check_update")


def gs_unscale_check_update_noalloc(grads: list[torch.Tensor], outs: list[torch.Tensor],
                                    scale: torch.Tensor, growth_tracker: torch.Tensor,
                                    found_inf: torch.Tensor, skipped: torch.Tensor | None = None,
                                    growth_factor: float = 2.0, backoff_factor: float = 0.5,
                                    growth_interval: int = 2000, stream=None) -> None:
    """The GradScaler step without any device allocation (for callers that
    cannot allocate): same results as gs_unscale_check_update, the list
    given on every call, the chunk table kept in the library's fixed device
    array."""
    if len(grads) != len(outs):
        raise ValueError("grads and outs differ in length")
    for g, o in zip(grads, outs):
        _contig(g, "grad")
        _contig(o, "out")
        if g.dtype != torch.float16 or o.dtype != torch.float32 or g.numel() != o.numel():
            raise ValueError("each grad must be float16 and its out float32 of equal numel")
    n = len(grads)
    gp = (ctypes.c_void_p * max(n, 1))(*[g.data_ptr() for g in grads])
    op = (ctypes.c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
    ne = (ctypes.c_int64 * max(n, 1))(*[g.numel() for g in grads])
    _check(_lib.gs_unscale_check_update_noalloc(gp, op, ne, n, _ptr(scale), _ptr(growth_tracker),
                                                _ptr(found_inf), _ptr(skipped), growth_factor,
                                                backoff_factor, growth_interval, _stream(stream)),
           "gs_unscale_check_update_noalloc")


def gs_noalloc_limits() -> tuple[int, int, int]:
    t, c, e = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.gs_noalloc_limits(ctypes.byref(t), ctypes.byref(c), ctypes.byref(e)),
           "gs_noalloc_limits")
    return t.value, c.value, e.value


def gs_unscale_check_update_norm(tlist: TensorList, scale: torch.Tensor,
                                 growth_tracker: torch.Tensor, found_inf: torch.Tensor,
                                 grad_norm: torch.Tensor, skipped: torch.Tensor | None = None,
                                 growth_factor: float = 2.0, backoff_factor: float = 0.5,
                                 growth_interval: int = 2000, stream=None) -> None:
    _check(_lib.gs_unscale_check_update_norm(tlist.handle, _ptr(scale), _ptr(growth_tracker),
                                             _ptr(found_inf), _ptr(skipped), growth_factor,
                                             backoff_factor, growth_interval, _ptr(grad_norm),
                                             _stream(stream)), "gs_unscale_check_update_norm")


class ParamList:
    """Owns a ``gs_param_list`` handle: fp32 master weights, optional bf16
    copies and fp32 gradients, tensor by tensor."""

    def __init__(self, master: list[torch.Tensor], grads: list[torch.Tensor],
                 master_bf16: list[torch.Tensor] | None = None):
        n = len(master)
        if len(grads) != n or (master_bf16 is not None and len(master_bf16) != n):
            raise ValueError("lists differ in length")
        for i in range(n):
            _contig(master[i], "master")
            _contig(grads[i], "grad")
            if master[i].dtype != torch.float32 or grads[i].dtype != torch.float32 or \
                    master[i].numel() != grads[i].numel():
                raise ValueError("master and grads must be float32 of equal numel")
            if master_bf16 is not None and (master_bf16[i].dtype != torch.bfloat16 or
                                            master_bf16[i].numel() != master[i].numel()):
                raise ValueError("master_bf16 must be bfloat16 of the same numel")
        self._keep = (list(master), list(grads), list(master_bf16 or []))
        k = max(n, 1)
        mp = (ctypes.c_void_p * k)(*[t.data_ptr() for t in master])
        gp = (ctypes.c_void_p * k)(*[t.data_ptr() for t in grads])
        bp = (ctypes.c_void_p * k)(*[t.data_ptr() for t in master_bf16]) if master_bf16 else None
        ne = (ctypes.c_int64 * k)(*[t.numel() for t in master])
        h = ctypes.c_void_p()
        _check(_lib.gs_param_list_create(mp, bp, gp, ne, n, ctypes.byref(h)), "gs_param_list_create")
        self.handle = h

    def close(self) -> None:
        if getattr(self, "handle", None):
            _lib.gs_param_list_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gs_param_list_create(master, grads, master_bf16=None) -> ParamList:
    return ParamList(master, grads, master_bf16)


def gs_master_update_sgd(plist: ParamList, lr: float, max_norm: float, grad_norm: torch.Tensor | None,
                         found_inf: torch.Tensor, stream=None) -> None:
    _check(_lib.gs_master_update_sgd(plist.handle, lr, max_norm, _ptr(grad_norm), _ptr(found_inf),
                                     _stream(stream)), "gs_master_update_sgd")


class AdamWList:
    """Owns a ``gs_adamw_list`` handle: fp32 master weights, gradients (all
    float32, bfloat16 or float16), both moments and optional bf16 copies,
    tensor by tensor.  Moments are float32 tensors, or uint8 E4M3 codes with
    float32 scales of ceil(numel / 128) values each."""

    def __init__(self, master: list[torch.Tensor], grads: list[torch.Tensor], m: list[torch.Tensor],
                 v: list[torch.Tensor], m_scale: list[torch.Tensor] | None = None,
                 v_scale: list[torch.Tensor] | None = None,
                 master_bf16: list[torch.Tensor] | None = None, decay: list[float] | None = None):
        n = len(master)
        for other in (grads, m, v, m_scale, v_scale, master_bf16, decay):
            if other is not None and len(other) != n:
                raise ValueError("lists differ in length")
        if (m_scale is None) != (v_scale is None):
            raise ValueError("m_scale and v_scale go together")
        mt = torch.float32 if m_scale is None else torch.uint8
        for i in range(n):
            k = master[i].numel()
            blocks = -(-k // 128)
            for t, name, dtype, numel in (
                    (master[i], "master", torch.float32, k), (grads[i], "grad", grads[0].dtype, k),
                    (m[i], "m", mt, k), (v[i], "v", mt, k),
                    (m_scale and m_scale[i], "m_scale", torch.float32, blocks),
                    (v_scale and v_scale[i], "v_scale", torch.float32, blocks),
                    (master_bf16 and master_bf16[i], "master_bf16", torch.bfloat16, k)):
                if t is None:
                    continue
                _contig(t, name)
                if t.dtype != dtype or t.numel() != numel:
                    raise ValueError(f"{name} {i} must be {dtype} with {numel} elements")
        self._keep = [list(t) for t in (master, grads, m, v, m_scale or [], v_scale or [],
                                        master_bf16 or [])]

        def ptrs(ts):
            return None if ts is None else (ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in ts])

        dk = None if decay is None else (ctypes.c_float * max(n, 1))(*decay)
        ne = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in master])
        h = ctypes.c_void_p()
        _check(_lib.gs_adamw_list_create(
            ptrs(master), ptrs(master_bf16), ptrs(grads),
            _DTYPES[grads[0].dtype] if n else GS_F32,
            GS_MOMENTS_F32 if m_scale is None else GS_MOMENTS_E4M3, ptrs(m), ptrs(v),
            ptrs(m_scale), ptrs(v_scale), dk, ne, n, ctypes.byref(h)), "gs_adamw_list_create")
        self.handle = h

    def close(self) -> None:
        if getattr(self, "handle", None):
            _lib.gs_adamw_list_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gs_adamw_list_create(master, grads, m, v, m_scale=None, v_scale=None, master_bf16=None,
                         decay=None) -> AdamWList:
    return AdamWList(master, grads, m, v, m_scale, v_scale, master_bf16, decay)


def gs_master_update_adamw(alist: AdamWList, step: torch.Tensor, found_inf: torch.Tensor, lr: float,
                           beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                           weight_decay: float = 0.01, max_norm: float = 0.0,
                           grad_norm: torch.Tensor | None = None, seed: int = 0,
                           stream=None) -> None:
    """step: int64 [1], the number of updates made so far (advanced on the
    device unless found_inf is set), this list's own; found_inf: int32 [1];
    grad_norm: float32 [1]."""
    # (_vector, _ptr and _check in line: small lists are bound by this call, and the
    # checks alone are 0.5 us of it)
    if (step is not None and (step.dtype is not _I64 or step.nbytes != 8) or
            found_inf is not None and (found_inf.dtype is not _I32 or found_inf.nbytes != 4) or
            grad_norm is not None and (grad_norm.dtype is not _F32 or grad_norm.nbytes != 4)):
        raise ValueError("step must be int64, found_inf int32 and grad_norm float32, of one element each")
    status = _lib.gs_master_update_adamw(
        alist.handle, lr, beta1, beta2, eps, weight_decay, max_norm,
        None if grad_norm is None else grad_norm.data_ptr(),
        None if found_inf is None else found_inf.data_ptr(),
        None if step is None else step.data_ptr(), seed, _stream(stream))
    if status != GS_OK:
        raise GsError(status, "gs_master_update_adamw")


class MuonList:
    """Owns a ``gs_muon_list`` handle: fp32 master matrices [rows, cols], their
    gradients (all float32, bfloat16 or float16), fp32 momenta and optional bf16
    copies, and the workspace of the step (8 to 12 bytes per element; rows are
    counted up to a multiple of 8 elements in it)."""

    def __init__(self, master: list[torch.Tensor], grads: list[torch.Tensor],
                 momentum: list[torch.Tensor], master_bf16: list[torch.Tensor] | None = None):
        n = len(master)
        for other in (grads, momentum, master_bf16):
            if other is not None and len(other) != n:
                raise ValueError("lists differ in length")
        for i in range(n):
            if master[i].dim() != 2:
                raise ValueError(f"master {i} must be a matrix")
            for t, name, dtype in ((master[i], "master", torch.float32), (grads[i], "grad", grads[0].dtype),
                                   (momentum[i], "momentum", torch.float32),
                                   (master_bf16 and master_bf16[i], "master_bf16", torch.bfloat16)):
                if t is None:
                    continue
                _contig(t, name)
                if t.dtype != dtype or t.shape != master[i].shape:
                    raise ValueError(f"{name} {i} must be {dtype} of shape {tuple(master[i].shape)}")
        self._keep = [list(t) for t in (master, grads, momentum, master_bf16 or [])]

        def ptrs(ts):
            return None if ts is None else (ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in ts])

        rows = (ctypes.c_int64 * max(n, 1))(*[t.shape[0] for t in master])
        cols = (ctypes.c_int64 * max(n, 1))(*[t.shape[1] for t in master])
        h = ctypes.c_void_p()
        _check(_lib.gs_muon_list_create(ptrs(master), ptrs(master_bf16), ptrs(grads),
                                        _DTYPES[grads[0].dtype] if n else GS_F32, ptrs(momentum), rows,
                                        cols, n, ctypes.byref(h)), "gs_muon_list_create")
        self.handle = h

    def close(self) -> None:
        if getattr(self, "handle", None):
            _lib.gs_muon_list_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gs_muon_list_create(master, grads, momentum, master_bf16=None) -> MuonList:
    return MuonList(master, grads, momentum, master_bf16)


def gs_master_update_muon(mlist: MuonList, found_inf: torch.Tensor, lr: float, momentum: float = 0.95,
                          weight_decay: float = 0.0, nesterov: bool = True, ns_steps: int = 5,
                          scale: str = "rms", max_norm: float = 0.0,
                          grad_norm: torch.Tensor | None = None, stream=None) -> None:
    """found_inf: int32 [1]; grad_norm: float32 [1]; scale: "rms" or "aspect"."""
    if (found_inf is not None and (found_inf.dtype is not _I32 or found_inf.nbytes != 4) or
            grad_norm is not None and (grad_norm.dtype is not _F32 or grad_norm.nbytes != 4)):
        raise ValueError("found_inf must be int32 and grad_norm float32, of one element each")
    _check(_lib.gs_master_update_muon(mlist.handle, lr, momentum, weight_decay, int(nesterov), ns_steps,
                                      _MUON_SCALES[scale], max_norm, _ptr(grad_norm), _ptr(found_inf),
                                      _stream(stream)), "gs_master_update_muon")


def gs_unscale_check_update_hysteresis(tlist: TensorList, scale: torch.Tensor,
                                       growth_tracker: torch.Tensor, hysteresis_state: torch.Tensor,
                                       found_inf: torch.Tensor, skipped: torch.Tensor | None = None,
                                       growth_factor: float = 2.0, backoff_factor: float = 0.5,
                                       window: int = 1000, hysteresis: int = 2,
                                       consecutive_hysteresis: bool = False, min_scale: float = 1.0,
                                       stream=None) -> None:
    _check(_lib.gs_unscale_check_update_hysteresis(
        tlist.handle, _ptr(scale), _ptr(growth_tracker), _ptr(hysteresis_state), _ptr(found_inf),
        _ptr(skipped), growth_factor, backoff_factor, window, hysteresis,
        int(consecutive_hysteresis), min_scale, _stream(stream)), "gs_unscale_check_update_hysteresis")


def fp8_quant_tensor_delayed(x: torch.Tensor, fmt, q: torch.Tensor, amax_history: torch.Tensor,
                             history_pos: torch.Tensor, scale_used: torch.Tensor, ws: torch.Tensor,
                             stream=None) -> None:
    _contig(x, "x")
    _check(_lib.fp8_quant_tensor_delayed(_ptr(x), _DTYPES[x.dtype], x.numel(), _FMTS[fmt], _ptr(q),
                                         _ptr(amax_history), amax_history.numel(), _ptr(history_pos),
                                         _ptr(scale_used), _ptr(ws), _stream(stream)),
           "fp8_quant_tensor_delayed")


def gs_scaler_state_get(scale: torch.Tensor, growth_tracker: torch.Tensor,
                        stream=None) -> tuple[float, int]:
    hs, ht = ctypes.c_float(), ctypes.c_int32()
    _check(_lib.gs_scaler_state_get(_ptr(scale), _ptr(growth_tracker), ctypes.byref(hs),
                                    ctypes.byref(ht), _stream(stream)), "gs_scaler_state_get")
    return hs.value, ht.value


def gs_scaler_state_set(scale: torch.Tensor, growth_tracker: torch.Tensor, h_scale: float,
                        h_growth_tracker: int, stream=None) -> None:
    _check(_lib.gs_scaler_state_set(_ptr(scale), _ptr(growth_tracker), h_scale, h_growth_tracker,
                                    _stream(stream)), "gs_scaler_state_set")


def fp8_quant_block(x: torch.Tensor, block_r: int, block_c: int, fmt, q: torch.Tensor,
                    scales: torch.Tensor, stream=None) -> None:
    """x: [R, C] bf16 / f16 / f32; q: uint8 [R, C]; scales: f32 [R/br, C/bc]."""
    _contig(x, "x")
    R, C = x.shape
    _check(_lib.fp8_quant_block(_ptr(x), _DTYPES[x.dtype], R, C, block_r, block_c, _FMTS[fmt],
                                _ptr(q), _ptr(scales), _stream(stream)), "fp8_quant_block")


def fp8_quant_tensor(x: torch.Tensor, fmt, q: torch.Tensor, scale: torch.Tensor,
                     ws: torch.Tensor, stream=None) -> None:
    _contig(x, "x")
    _check(_lib.fp8_quant_tensor(_ptr(x), _DTYPES[x.dtype], x.numel(), _FMTS[fmt], _ptr(q),
                                 _ptr(scale), _ptr(ws), _stream(stream)), "fp8_quant_tensor")


def fp8_dequant(q: torch.Tensor, scales: torch.Tensor, block_r: int, block_c: int, fmt,
                y: torch.Tensor, stream=None) -> None:
    """q: uint8 [R, C]; y: f32 or bf16 [R, C]; (block_r, block_c) = (1,128),
    (128,128) or (R, C) for one per-tensor scale."""
    _contig(q, "q")
    R, C = q.shape
    _check(_lib.fp8_dequant(_ptr(q), _ptr(scales), R, C, block_r, block_c, _FMTS[fmt],
                            _DTYPES[y.dtype], _ptr(y), _stream(stream)), "fp8_dequant")


def fp8_quant_mx(x: torch.Tensor, fmt, q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """x: [R, C] (C % 32 == 0) bf16 / f16 / f32; q: uint8 [R, C]; scales: uint8 [R, C/32]."""
    _contig(x, "x")
    R, C = x.shape
    _check(_lib.fp8_quant_mx(_ptr(x), _DTYPES[x.dtype], R, C, _FMTS[fmt], _ptr(q), _ptr(scales),
                             _stream(stream)), "fp8_quant_mx")


def fp8_dequant_mx(q: torch.Tensor, scales: torch.Tensor, fmt, y: torch.Tensor, stream=None) -> None:
    _contig(q, "q")
    R, C = q.shape
    _check(_lib.fp8_dequant_mx(_ptr(q), _ptr(scales), R, C, _FMTS[fmt], _DTYPES[y.dtype], _ptr(y),
                               _stream(stream)), "fp8_dequant_mx")


def fp8_gemm_block_scaled(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor,
                          fmt, d: torch.Tensor, stream=None, fmt_b=None) -> None:
    """d[M, N] = block-scaled qa[M, K] @ qb[N, K]^T, promoted to fp32 every
    128 of K. qa is in format `fmt`, qb in `fmt_b` (default: the same)."""
    fmt_b = fmt if fmt_b is None else fmt_b
    for t, name in ((qa, "qa"), (sa, "sa"), (qb, "qb"), (sb, "sb"), (d, "d")):
        _contig(t, name)
    M, K = qa.shape
    N = qb.shape[0]
    if qb.shape[1] != K or tuple(d.shape) != (M, N):
        raise ValueError(f"fp8_gemm_block_scaled: shapes qa {tuple(qa.shape)}, "
                         f"qb {tuple(qb.shape)}, d {tuple(d.shape)}")
    _check(_lib.fp8_gemm_block_scaled(_ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), M, N, K, _FMTS[fmt],
                                      _FMTS[fmt_b], _DTYPES[d.dtype], _ptr(d), _stream(stream)),
           "fp8_gemm_block_scaled")


def _rows(t: torch.Tensor, name: str, shape=None) -> int:
    """The distance of two rows of a [R, C] tensor, in elements."""
    st, sh = t.stride(), t.shape
    if len(st) != 2 or (st[1] != 1 and sh[1] > 1):
        raise ValueError(f"{name} must be [rows, columns] with adjacent columns")
    if shape is not None and sh != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return st[0] if sh[0] > 1 else max(sh[1], 1)


def _vector(t: torch.Tensor | None, name: str, n: int, dtype: torch.dtype) -> int | None:
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of {n} elements and {dtype}")
    return t.data_ptr()


def gs_layernorm_fwd(x: torch.Tensor, gamma: torch.Tensor | None, beta: torch.Tensor | None,
                     y: torch.Tensor, mean: torch.Tensor | None = None,
                     rstd: torch.Tensor | None = None, eps: float = 1e-5, stream=None) -> None:
    """x, y: [R, C] of one type (rows may be apart); gamma, beta: [C], float32
    or x's type, or None; mean, rstd: float32 [R] or None."""
    shape = x.shape
    ldx, ldy = _rows(x, "x"), _rows(y, "y", shape)
    R, C = shape
    if y.dtype != x.dtype:
        raise ValueError("y must have the type of x")
    w = gamma if gamma is not None else beta
    wt = torch.float32 if w is None else w.dtype
    _check(_lib.gs_layernorm_fwd(x.data_ptr(), ldx, _DTYPES[x.dtype], R, C,
                                 _vector(gamma, "gamma", C, wt), _vector(beta, "beta", C, wt),
                                 _DTYPES[wt], eps, y.data_ptr(), ldy,
                                 _vector(mean, "mean", R, torch.float32),
                                 _vector(rstd, "rstd", R, torch.float32), _stream(stream)),
           "gs_layernorm_fwd")


def gs_layernorm_ws_bytes(rows: int, cols: int) -> int:
    return int(_lib.gs_layernorm_ws_bytes(rows, cols))


def gs_layernorm_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor | None,
                     mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                     dgamma: torch.Tensor | None = None, dbeta: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None) -> None:
    """dy, x, dx: [R, C] of one type; dgamma, dbeta: [C] of one type (float32,
    bfloat16 or float16) or None; ws: gs_layernorm_ws_bytes(R, C) bytes."""
    shape = x.shape
    ldx, lddy, lddx = _rows(x, "x"), _rows(dy, "dy", shape), _rows(dx, "dx", shape)
    R, C = shape
    if dy.dtype != x.dtype or dx.dtype != x.dtype:
        raise ValueError("dy and dx must have the type of x")
    wt = torch.float32 if gamma is None else gamma.dtype
    d = dgamma if dgamma is not None else dbeta
    dt = torch.float32 if d is None else d.dtype
    if ws is not None and (not ws.is_contiguous() or
                           ws.numel() * ws.element_size() < gs_layernorm_ws_bytes(R, C)):
        raise ValueError("ws must be contiguous, of gs_layernorm_ws_bytes(R, C) bytes at least")
    _check(_lib.gs_layernorm_bwd(_ptr(dy), lddy, _ptr(x), ldx, _DTYPES[x.dtype], R, C,
                                 _vector(gamma, "gamma", C, wt), _DTYPES[wt],
                                 _vector(mean, "mean", R, torch.float32),
                                 _vector(rstd, "rstd", R, torch.float32), _ptr(dx), lddx,
                                 _vector(dgamma, "dgamma", C, dt), _vector(dbeta, "dbeta", C, dt),
                                 _DTYPES[dt], _ptr(ws), _stream(stream)), "gs_layernorm_bwd")


def gs_token_logprob(logits: torch.Tensor, targets: torch.Tensor | None,
                     logprob: torch.Tensor | None, lse: torch.Tensor | None = None,
                     entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                     top_logprob: torch.Tensor | None = None, stream=None) -> None:
    """logits: [R, V] (rows may be apart); targets: int64 [R]; logprob, lse,
    entropy: float32 [R]; top_ids: int32 [R, k], top_logprob: float32 [R, k].
    Every output but at least one may be None."""
    ld = _rows(logits, "logits")
    R, V = logits.shape
    if (top_ids is None) != (top_logprob is None):
        raise ValueError("top_ids and top_logprob go together")
    k = 0
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape[0] != R:
            raise ValueError("top_ids must be [rows, k]")
        k = top_ids.shape[1]
    f32 = torch.float32
    _check(_lib.gs_token_logprob(_ptr(logits), ld, _DTYPES[logits.dtype], R, V,
                                 _vector(targets, "targets", R, torch.int64),
                                 _vector(logprob, "logprob", R, f32), _vector(lse, "lse", R, f32),
                                 _vector(entropy, "entropy", R, f32), k,
                                 _vector(top_ids, "top_ids", R * k, torch.int32),
                                 _vector(top_logprob, "top_logprob", R * k, f32), _stream(stream)),
           "gs_token_logprob")


def gs_token_logprob_bwd(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                         dlogprob: torch.Tensor, dlogits: torch.Tensor,
                         entropy: torch.Tensor | None = None, dentropy: torch.Tensor | None = None,
                         loss_scale: torch.Tensor | None = None, stream=None) -> None:
    """dlogits: [R, V], any of the three types, or the logits themselves; lse
    and entropy as gs_token_logprob wrote them; loss_scale: float32 [1]."""
    ld, ld_out = _rows(logits, "logits"), _rows(dlogits, "dlogits", logits.shape)
    R, V = logits.shape
    f32 = torch.float32
    _check(_lib.gs_token_logprob_bwd(_ptr(logits), ld, _DTYPES[logits.dtype], R, V,
                                     _vector(targets, "targets", R, torch.int64),
                                     _vector(lse, "lse", R, f32),
                                     _vector(dlogprob, "dlogprob", R, f32),
                                     _vector(entropy, "entropy", R, f32),
                                     _vector(dentropy, "dentropy", R, f32),
                                     _vector(loss_scale, "loss_scale", 1, f32), _ptr(dlogits),
                                     ld_out, _DTYPES[dlogits.dtype], _stream(stream)),
           "gs_token_logprob_bwd")


_WS_BYTES = gs_ws_bytes()


def fp4_scale_bytes(rows: int, cols: int, fmt) -> int:
    """Bytes of the scales of a [rows, cols] 4-bit tensor (tiles of 512 bytes)."""
    return int(_lib.fp4_scale_bytes(rows, cols, _FMTS4[fmt]))


def _codes4(q: torch.Tensor, scales: torch.Tensor, name: str, R: int, C: int, fmt: int) -> None:
    """Checks that q holds the codes and scales the scales of [R, C] values."""
    if q.dtype is not torch.uint8 or q.shape != (R, C // 2) or not q.is_contiguous():
        raise ValueError(f"{name} must be contiguous uint8 [{R}, {C // 2}]")
    n = -(-R // 128) * -(-C // (64 if fmt == GS_NVFP4 else 128)) * 512
    if scales.dtype is not torch.uint8 or scales.numel() != n or not scales.is_contiguous():
        raise ValueError(f"the scales of {name} must be contiguous uint8, of {n} bytes")


def fp4_quant(x: torch.Tensor, fmt, q: torch.Tensor | None, scales: torch.Tensor | None,
              tensor_scale: torch.Tensor | None = None, ws: torch.Tensor | None = None,
              qt: torch.Tensor | None = None, scales_t: torch.Tensor | None = None, stream=None) -> None:
    """x: [R, C] bf16 / f16 / f32 (rows may be apart); q: uint8 [R, C/2], scales:
    uint8, fp4_scale_bytes(R, C) of them; qt: uint8 [C, R/2] and scales_t
    (fp4_scale_bytes(C, R)) for the transpose; either pair may be None.
    tensor_scale ("nvfp4"): float32 [1], formed from x and written where ws
    (gs_ws_bytes() bytes) is given, else read."""
    ldx, f = _rows(x, "x"), _FMTS4[fmt]
    R, C = x.shape
    if (q is None) != (scales is None) or (qt is None) != (scales_t is None):
        raise ValueError("codes and scales go together")
    if q is not None:
        _codes4(q, scales, "q", R, C, f)
    if qt is not None:
        _codes4(qt, scales_t, "qt", C, R, f)
    if ws is not None and (not ws.is_contiguous() or ws.nbytes < _WS_BYTES):
        raise ValueError("ws must be contiguous, of gs_ws_bytes() bytes at least")
    _check(_lib.fp4_quant(_ptr(x), ldx, _DTYPES[x.dtype], R, C, f, _ptr(q), _ptr(scales), _ptr(qt),
                          _ptr(scales_t), _vector(tensor_scale, "tensor_scale", 1, _F32), _ptr(ws),
                          _stream(stream)), "fp4_quant")


def fp4_dequant(q: torch.Tensor, scales: torch.Tensor, fmt, y: torch.Tensor,
                tensor_scale: torch.Tensor | None = None, stream=None) -> None:
    """y: [R, C], any of the three types (rows may be apart), from q [R, C/2]."""
    ldy, f = _rows(y, "y"), _FMTS4[fmt]
    R, C = y.shape
    _codes4(q, scales, "q", R, C, f)
    _check(_lib.fp4_dequant(_ptr(q), _ptr(scales), _vector(tensor_scale, "tensor_scale", 1, _F32), R, C,
                            f, _DTYPES[y.dtype], _ptr(y), ldy, _stream(stream)), "fp4_dequant")


def fp4_gemm_block_scaled(qa: torch.Tensor, sa: torch.Tensor, qb: torch.Tensor, sb: torch.Tensor, fmt,
                          d: torch.Tensor, ta: torch.Tensor | None = None,
                          tb: torch.Tensor | None = None, stream=None) -> None:
    """d[M, N] = ta tb (qa[M, K/2] with scales sa) @ (qb[N, K/2] with sb)^T;
    d float32 or bfloat16, rows may be apart; ta, tb: float32 [1] ("nvfp4")."""
    ldd, f = _rows(d, "d"), _FMTS4[fmt]
    M, N = d.shape
    K = 2 * qa.shape[-1]
    _codes4(qa, sa, "qa", M, K, f)
    _codes4(qb, sb, "qb", N, K, f)
    _check(_lib.fp4_gemm_block_scaled(qa.data_ptr(), sa.data_ptr(), _vector(ta, "ta", 1, _F32),
                                      qb.data_ptr(), sb.data_ptr(), _vector(tb, "tb", 1, _F32), M, N, K,
                                      f, _DTYPES[d.dtype], d.data_ptr(), ldd, _stream(stream)),
           "fp4_gemm_block_scaled")


def gs_policy_loss_ws_bytes(tokens: int, seqs: int = 1) -> int:
    return int(_lib.gs_policy_loss_ws_bytes(tokens, seqs))


def gs_policy_loss(logprob: torch.Tensor, old_logprob: torch.Tensor, advantages: torch.Tensor,
                   loss: torch.Tensor, ws: torch.Tensor, dlogprob: torch.Tensor | None = None,
                   stats: torch.Tensor | None = None, ref_logprob: torch.Tensor | None = None,
                   targets: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                   dloss: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                   dual_clip: float = 0.0, kl_coef: float = 0.0, reduction: str = "token",
                   stream=None, per_sequence: bool | None = None) -> None:
    """logprob, old_logprob, ref_logprob, dlogprob: float32 [T]; advantages:
    float32 [T] or [S] (per_sequence says which; unless said their length does,
    [T] where T == S); targets: int64 [T] (negative: the token does not
    count); seq_offsets: int64 [S + 1]; loss, dloss: float32 [1]; stats:
    float32 [4] (tokens, mean ratio, held fraction, mean divergence); ws:
    gs_policy_loss_ws_bytes(T, S) bytes; reduction: "token", "sequence" or
    "sum"."""
    T = logprob.numel()
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    n = advantages.numel()
    if per_sequence is not None and n != (S if per_sequence else T):
        raise ValueError("advantages must be one per sequence" if per_sequence else "advantages must be one per token")
    if not ws.is_contiguous() or ws.nbytes < _lib.gs_policy_loss_ws_bytes(T, S):
        raise ValueError("ws must be contiguous, of gs_policy_loss_ws_bytes(T, S) bytes at least")
    status = _lib.gs_policy_loss(
        _vector(logprob, "logprob", T, _F32), _vector(old_logprob, "old_logprob", T, _F32),
        _vector(ref_logprob, "ref_logprob", T, _F32), _vector(advantages, "advantages", n, _F32),
        -n if per_sequence else n, _vector(targets, "targets", T, _I64), T, _vector(seq_offsets, "seq_offsets", S + 1, _I64), S,
        clip_low, clip_high, dual_clip, kl_coef, _REDUCTIONS[reduction], _vector(dloss, "dloss", 1, _F32),
        _vector(loss, "loss", 1, _F32), _vector(stats, "stats", 4, _F32),
        _vector(dlogprob, "dlogprob", T, _F32), ws.data_ptr(), _stream(stream))
    if status != GS_OK:
        raise GsError(status, "gs_policy_loss")


def gs_test_set_stall(on: bool) -> None:
    """Test hook: the block-scaled FP8 and 4-bit products and the products of
    gs_master_update_muon issue no TMA loads while on, so their bounded waits
    run out and they report GS_ERR_TIMEOUT."""
    _check(_lib.gs_test_set_stall(1 if on else 0), "gs_test_set_stall")


def gs_test_adamw_root(v: torch.Tensor, r: torch.Tensor, stream=None) -> None:
    """Test hook: r = sqrt(v) as the 8-bit AdamW step forms it; float32, of one
    even length."""
    n = v.numel()
    _check(_lib.gs_test_adamw_root(_vector(v, "v", n, torch.float32), _vector(r, "r", n, torch.float32),
                                   n, _stream(stream)), "gs_test_adamw_root")


def gs_device_status(stream=None) -> int:
    v = ctypes.c_int32()
    _check(_lib.gs_device_status(ctypes.byref(v), _stream(stream)), "gs_device_status")
    return v.value
