"""ctypes binding of libpoetx (include/poetx.h).

Argument marshalling only: each function below has the name of the C entry point
it calls and forwards raw device pointers, sizes and the HIP stream.  Every step
of the layer runs in the library's HIP kernels; there is no fallback path, and a
missing or unloadable library raises.

Tensors are torch tensors on the GPU (torch provides device memory and
streams).  bfloat16 data may be passed as torch.bfloat16 or as 16-bit integer
tensors holding the bit patterns.
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# POETX_LIBRARY names another build of the library (e.g. to compare two builds in one process tree)
LIB_PATH = os.environ.get("POETX_LIBRARY") or os.path.join(HERE, "libpoetx.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "poetx.h")

POETX_OK, POETX_E_NULL, POETX_E_SHAPE, POETX_E_DTYPE, POETX_E_WORKSPACE, POETX_E_PERM, POETX_E_HIP, POETX_E_UNSUPPORTED = range(8)
POETX_F32, POETX_BF16, POETX_I8 = 0, 1, 2
POETX_OP_CNP, POETX_OP_FWD, POETX_OP_BWD, POETX_OP_MERGE = 0, 1, 2, 3
POETX_KC_NONE, POETX_KC_GEMM, POETX_KC_APPLY, POETX_KC_DGRAD, POETX_KC_CNP, POETX_KC_PERMUTE, POETX_KC_OPTIM = range(7)

DTYPES = {"f32": POETX_F32, "bf16": POETX_BF16, "i8": POETX_I8}
# what the forward saves: H and Xt; Xt only (H recomputed from it); Xt only (H taken back from Y)
POETX_XFAST, POETX_XMEM, POETX_XOUT = 0, 1, 2
POETX_MAX_SIDES = 64  # most sides one batched call accepts
POETX_MAX_GROUP = 8  # most linears one group call accepts
MODES = {"xfast": POETX_XFAST, "xmem": POETX_XMEM, "xout": POETX_XOUT}


class PoetxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libpoetx status {status}: {msg}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [
        ("m", ctypes.c_int32),
        ("n", ctypes.c_int32),
        ("b", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
        ("w_dtype", ctypes.c_int32),
        ("mode", ctypes.c_int32),
    ]


POETX_SPO_BLOCK, POETX_SPO_FULL = 0, 1
SPO_KINDS = {"block": POETX_SPO_BLOCK, "full": POETX_SPO_FULL}


class SpoDesc(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int32),
        ("b", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
    ]


class GradSide(ctypes.Structure):
    _fields_ = [
        ("A", ctypes.c_void_p),
        ("lda", ctypes.c_int64),
        ("B", ctypes.c_void_p),
        ("ldb", ctypes.c_int64),
        ("d", ctypes.c_int32),
    ]


class FwdCall(ctypes.Structure):
    _fields_ = [
        ("desc", ctypes.POINTER(LayerDesc)),
        ("X", ctypes.c_void_p),
        ("perm_R", ctypes.c_void_p),
        ("perm_P", ctypes.c_void_p),
        ("Wt", ctypes.c_void_p),
        ("g_R", ctypes.c_void_p),
        ("g_P", ctypes.c_void_p),
        ("Y", ctypes.c_void_p),
        ("H_save", ctypes.c_void_p),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t),
    ]


class BwdCall(ctypes.Structure):
    _fields_ = [
        ("desc", ctypes.POINTER(LayerDesc)),
        ("Y", ctypes.c_void_p),
        ("dZ", ctypes.c_void_p),
        ("perm_R", ctypes.c_void_p),
        ("perm_P", ctypes.c_void_p),
        ("Wt", ctypes.c_void_p),
        ("g_R", ctypes.c_void_p),
        ("g_P", ctypes.c_void_p),
        ("H_save", ctypes.c_void_p),
        ("dX", ctypes.c_void_p),
        ("ws", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t),
    ]


POETX_NORM_LAYER, POETX_NORM_RMS = 0, 1
NORM_KINDS = {"layer": POETX_NORM_LAYER, "rms": POETX_NORM_RMS}


class NormDesc(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


POETX_ROPE_HALF, POETX_ROPE_PAIRS = 0, 1
ROPE_LAYOUTS = {"half": POETX_ROPE_HALF, "pairs": POETX_ROPE_PAIRS}
POETX_ROPE_NONE, POETX_ROPE_LINEAR, POETX_ROPE_BASE, POETX_ROPE_BANDS, POETX_ROPE_RAMP = range(5)
ROPE_SCALINGS = {"none": POETX_ROPE_NONE, "linear": POETX_ROPE_LINEAR, "base": POETX_ROPE_BASE,
                 "bands": POETX_ROPE_BANDS, "ramp": POETX_ROPE_RAMP}


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
    ]


class RopeParams(ctypes.Structure):
    _fields_ = [
        ("base", ctypes.c_double),
        ("scaling", ctypes.c_int32),
        ("factor", ctypes.c_double),
        ("original", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
    ]


class AttnDesc(ctypes.Structure):
    _fields_ = [
        ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class LogpDesc(ctypes.Structure):
    _fields_ = [
        ("vocab", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
        ("top", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class AdamParams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("t", ctypes.c_int64),
    ]


class NsParams(ctypes.Structure):
    _fields_ = [
        ("steps", ctypes.c_int32),
        ("a", ctypes.c_float),
        ("b", ctypes.c_float),
        ("c", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("rms", ctypes.c_float),
    ]


class MuonParams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("nesterov", ctypes.c_int32),
        ("ns", NsParams),
    ]


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_SIG = {
    "poetx_version": (ctypes.c_char_p, []),
    "poetx_last_error": (ctypes.c_char_p, []),
    "poetx_packed_len": (ctypes.c_int64, [ctypes.c_int32]),
    "poetx_g_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    "poetx_weight_bytes": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc)]),
    "poetx_saved_bytes": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc), ctypes.c_int64]),
    "poetx_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc), ctypes.c_int64, ctypes.c_int32]),
    "poetx_perm_from_seed": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]),
    "poetx_cnp_build": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, ctypes.c_size_t, _P]),
    "poetx_cnp_build_noalloc": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "poetx_premerge": (ctypes.c_int, [ctypes.POINTER(LayerDesc), _P, ctypes.c_int64, _P, _P, _P, _P, _P]),
    "poetx_linear_fwd": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), ctypes.c_int64, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    ),
    "poetx_linear_bwd": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), ctypes.c_int64] + [_P] * 14 + [ctypes.c_size_t, _P],
    ),
    "poetx_timer_enable": (ctypes.c_int, [ctypes.c_int32]),
    "poetx_timer_read": (
        ctypes.c_int,
        [ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
         ctypes.POINTER(ctypes.c_double)],
    ),
    "poetx_merge_reinit": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), _P, _P, _P, _P, _P, _P, _P, ctypes.c_uint64, ctypes.c_uint64, _P, ctypes.c_size_t, _P],
    ),
    "poetx_cnp_batch_workspace_size": (
        ctypes.c_size_t, [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, ctypes.c_int32]
    ),
    "poetx_cnp_build_batch": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, ctypes.c_int32,
         ctypes.POINTER(_P), _P, ctypes.c_size_t, _P],
    ),
    "poetx_cnp_grad_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    "poetx_linear_bwd_dx": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), ctypes.c_int64] + [_P] * 12 + [ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_size_t, _P],
    ),
    "poetx_cnp_backward_batch": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, ctypes.c_int32, _P,
         ctypes.c_size_t, ctypes.POINTER(_P), _P],
    ),
    "poetx_cnp_backward_batch_reuse": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, ctypes.c_int32, _P,
         ctypes.c_size_t, _P, ctypes.c_size_t, ctypes.POINTER(_P), _P],
    ),
    "poetx_linear_bwd_dx_sides": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), ctypes.c_int64] + [_P] * 9 + [ctypes.POINTER(GradSide), _P, ctypes.c_size_t, _P],
    ),
    "poetx_linear_fwd_group": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(FwdCall), ctypes.c_int64, _P]),
    "poetx_linear_bwd_dx_group": (
        ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(BwdCall), ctypes.c_int64, ctypes.POINTER(GradSide), _P]
    ),
    "poetx_block_grads_workspace_size": (
        ctypes.c_size_t, [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
    ),
    "poetx_block_grads_batch": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(GradSide), ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_size_t,
         _P, ctypes.c_size_t, _P],
    ),
    "poetx_spo_saved_bytes": (ctypes.c_size_t, [ctypes.POINTER(SpoDesc), ctypes.c_int64]),
    "poetx_spo_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(SpoDesc), ctypes.c_int64, ctypes.c_int32]),
    "poetx_spo_fwd": (ctypes.c_int, [ctypes.POINTER(SpoDesc), ctypes.c_int64] + [_P] * 6 + [ctypes.c_size_t, _P]),
    "poetx_spo_bwd": (ctypes.c_int, [ctypes.POINTER(SpoDesc), ctypes.c_int64] + [_P] * 8 + [ctypes.c_size_t, _P]),
    "poetx_fold_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc), ctypes.c_int32, ctypes.POINTER(SpoDesc)]),
    "poetx_fold_factor": (
        ctypes.c_int,
        [ctypes.POINTER(LayerDesc), ctypes.c_int32, ctypes.POINTER(SpoDesc), _P, _P, _P, _P, ctypes.c_int64, _P,
         ctypes.c_size_t, _P],
    ),
    "poetx_store_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc)]),
    "poetx_store_weight": (ctypes.c_int, [ctypes.POINTER(LayerDesc), _P, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P]),
    "poetx_wc_state_bytes": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc), ctypes.c_int64]),
    "poetx_wc_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LayerDesc), ctypes.c_int64, ctypes.c_int32]),
    "poetx_wc_fwd": (ctypes.c_int, [ctypes.POINTER(LayerDesc), ctypes.c_int64] + [_P] * 9 + [ctypes.c_size_t, _P]),
    "poetx_wc_bwd": (ctypes.c_int, [ctypes.POINTER(LayerDesc), ctypes.c_int64] + [_P] * 12 + [ctypes.c_size_t, _P]),
    "poetx_muon_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]),
    "poetx_muon_step_batch": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int32),
         ctypes.c_int32, ctypes.POINTER(MuonParams), _P, ctypes.c_size_t, _P],
    ),
    "poetx_orthogonalize_workspace_size": (
        ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    ),
    "poetx_orthogonalize": (
        ctypes.c_int,
        [ctypes.c_int32] * 4 + [_P, ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_int64,
                                ctypes.POINTER(NsParams), _P, ctypes.c_size_t, _P],
    ),
    "poetx_norm_stats_bytes": (ctypes.c_size_t, [ctypes.POINTER(NormDesc), ctypes.c_int64]),
    "poetx_norm_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(NormDesc), ctypes.c_int64]),
    "poetx_norm_fwd": (
        ctypes.c_int,
        [ctypes.POINTER(NormDesc), ctypes.c_int64, _P, ctypes.c_int64, _P, ctypes.c_int64, _P, _P, _P, ctypes.c_int64, _P,
         ctypes.c_int64, _P, _P],
    ),
    "poetx_norm_bwd": (
        ctypes.c_int,
        [ctypes.POINTER(NormDesc), ctypes.c_int64, _P, ctypes.c_int64, _P, ctypes.c_int64, _P, _P, _P, ctypes.c_int64, _P,
         ctypes.c_int64, _P, _P, _P, ctypes.c_size_t, _P],
    ),
    "poetx_rope_freqs": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(RopeParams), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_float)],
    ),
    "poetx_rope": (
        ctypes.c_int,
        [ctypes.POINTER(RopeDesc), ctypes.c_int64, _P, _P, ctypes.c_float, ctypes.c_int32, ctypes.c_int32,
         ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(_P),
         ctypes.POINTER(ctypes.c_int64), _P],
    ),
    "poetx_attn_workspace_size": (
        ctypes.c_size_t,
        [ctypes.POINTER(AttnDesc), ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32],
    ),
    "poetx_attn_fwd": (
        ctypes.c_int,
        [ctypes.POINTER(AttnDesc), ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, _P, _P] + [_P, ctypes.c_int64] * 4
        + [_P, _P, ctypes.c_size_t, _P],
    ),
    "poetx_attn_bwd": (
        ctypes.c_int,
        [ctypes.POINTER(AttnDesc), ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, _P, _P] + [_P, ctypes.c_int64] * 5
        + [_P] + [_P, ctypes.c_int64] * 3 + [_P, ctypes.c_size_t, _P],
    ),
    "poetx_logp_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(LogpDesc), ctypes.c_int64]),
    "poetx_logp_fwd": (
        ctypes.c_int,
        [ctypes.POINTER(LogpDesc), ctypes.c_int64, _P, ctypes.c_int64] + [_P] * 7 + [ctypes.c_size_t, _P],
    ),
    "poetx_logp_bwd": (
        ctypes.c_int,
        [ctypes.POINTER(LogpDesc), ctypes.c_int64, _P, ctypes.c_int64] + [_P] * 6 + [ctypes.c_int64, _P],
    ),
    "poetx_adam_step_batch": (
        ctypes.c_int,
        [ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P),
         ctypes.POINTER(_P), ctypes.POINTER(AdamParams), _P],
    ),
}


def lib() -> ctypes.CDLL:
    """Load libpoetx.so (after torch, so that both share one HIP runtime)."""
    global _lib
    if _lib is None:
        try:
            import torch  # noqa: F401  (loads the HIP runtime the library must share)
        except ImportError:
            pass
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run orthogonal_reparameterized_cnp_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIG.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_symbols() -> list:
    """Names of the functions include/poetx.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]+?\b(poetx_\w+)\s*\(", text, re.M)))


def _check(st: int):
    if st != POETX_OK:
        raise PoetxError(st, lib().poetx_last_error().decode())


def _ptr(t) -> Optional[int]:
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_stream() -> int:
    """The current stream's handle.  The first call picks torch's raw accessor where it has one: building the Stream
    object that torch.cuda.current_stream() returns costs more than the rest of a call's marshalling."""
    global _current_stream
    import torch

    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    torch.cuda.current_stream()  # initialises the GPU, or raises
    _current_stream = (lambda: raw(dev())) if raw and dev else (lambda: torch.cuda.current_stream().cuda_stream)
    return _current_stream()


def desc(m: int, n: int, b: int, act: str, w: str, mode: str = "xfast") -> LayerDesc:
    return LayerDesc(m, n, b, DTYPES[act], DTYPES[w], MODES[mode])


# ---------------------------------------------------------------- helpers ---
def poetx_version() -> str:
    return lib().poetx_version().decode()


def poetx_last_error() -> str:
    return lib().poetx_last_error().decode()


def poetx_packed_len(b: int) -> int:
    return lib().poetx_packed_len(b)


def poetx_g_bytes(d: int, b: int, dtype: int) -> int:
    return lib().poetx_g_bytes(d, b, dtype)


def poetx_weight_bytes(dsc: LayerDesc) -> int:
    return lib().poetx_weight_bytes(ctypes.byref(dsc))


def poetx_saved_bytes(dsc: LayerDesc, T: int) -> int:
    return lib().poetx_saved_bytes(ctypes.byref(dsc), T)


def poetx_workspace_size(dsc: LayerDesc, T: int, op: int) -> int:
    return lib().poetx_workspace_size(ctypes.byref(dsc), T, op)


def poetx_perm_from_seed(seed: int, d: int):
    import numpy as np

    out = np.empty(d, dtype=np.int32)
    _check(lib().poetx_perm_from_seed(seed, d, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))
    return out


def poetx_timer_enable(kernel_class: int):
    _check(lib().poetx_timer_enable(kernel_class))


def poetx_timer_read():
    """(launches, total_ms, flops, bytes) of the enabled class since the last read."""
    n, ms, fl, by = ctypes.c_int64(), ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    _check(lib().poetx_timer_read(ctypes.byref(n), ctypes.byref(ms), ctypes.byref(fl), ctypes.byref(by)))
    return n.value, ms.value, fl.value, by.value


# ------------------------------------------------------------- the calls ---
def poetx_cnp_build(q, d: int, b: int, dtype: int, g, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_cnp_build(_ptr(q), d, b, dtype, _ptr(g), _ptr(ws), ws_bytes, _stream(stream)))


def poetx_cnp_build_noalloc(q, d: int, b: int, dtype: int, g, stream=None):
    _check(lib().poetx_cnp_build_noalloc(_ptr(q), d, b, dtype, _ptr(g), _stream(stream)))


def poetx_premerge(dsc: LayerDesc, W0, ld_w0: int, w0_scale, perm_R, perm_P, Wt, stream=None):
    _check(
        lib().poetx_premerge(
            ctypes.byref(dsc), _ptr(W0), ld_w0, _ptr(w0_scale), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _stream(stream)
        )
    )


def poetx_linear_fwd(dsc: LayerDesc, T: int, X, perm_R, perm_P, Wt, g_R, g_P, Y, H_save, ws, ws_bytes: int, stream=None):
    _check(
        lib().poetx_linear_fwd(
            ctypes.byref(dsc), T, _ptr(X), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _ptr(g_R), _ptr(g_P), _ptr(Y),
            _ptr(H_save), _ptr(ws), ws_bytes, _stream(stream),
        )
    )


def poetx_linear_bwd(dsc: LayerDesc, T: int, Y, dZ, perm_R, perm_P, Wt, g_R, g_P, q_R, q_P, H_save, dX, dq_R, dq_P,
                     ws, ws_bytes: int, stream=None):
    _check(
        lib().poetx_linear_bwd(
            ctypes.byref(dsc), T, _ptr(Y), _ptr(dZ), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _ptr(g_R), _ptr(g_P),
            _ptr(q_R), _ptr(q_P), _ptr(H_save), _ptr(dX), _ptr(dq_R), _ptr(dq_P), _ptr(ws), ws_bytes, _stream(stream),
        )
    )


def poetx_merge_reinit(dsc: LayerDesc, Wt, perm_R, perm_P, g_R, g_P, q_R, q_P, seed_R: int, seed_P: int, ws,
                       ws_bytes: int, stream=None):
    _check(
        lib().poetx_merge_reinit(
            ctypes.byref(dsc), _ptr(Wt), _ptr(perm_R), _ptr(perm_P), _ptr(g_R), _ptr(g_P), _ptr(q_R), _ptr(q_P),
            seed_R & ((1 << 64) - 1), seed_P & ((1 << 64) - 1), _ptr(ws), ws_bytes, _stream(stream),
        )
    )


# ------------------------------------------------- batched CNP (one layer) ---
def _ptr_array(ts):
    return (_P * len(ts))(*[_ptr(t) for t in ts])


def _i32_array(xs):
    return (ctypes.c_int32 * len(xs))(*xs)


def poetx_cnp_batch_workspace_size(d, b: int, dtype: int) -> int:
    return lib().poetx_cnp_batch_workspace_size(len(d), _i32_array(d), b, dtype)


def poetx_cnp_build_batch(q, d, b: int, dtype: int, g, ws, ws_bytes: int, stream=None):
    """q, d, g: per-side lists (device tensors / ints), marshalled into host arrays."""
    _check(lib().poetx_cnp_build_batch(len(d), _ptr_array(q), _i32_array(d), b, dtype, _ptr_array(g), _ptr(ws),
                                       ws_bytes, _stream(stream)))


def poetx_cnp_grad_bytes(blocks: int, b: int, dtype: int) -> int:
    return lib().poetx_cnp_grad_bytes(blocks, b, dtype)


def poetx_linear_bwd_dx(dsc: LayerDesc, T: int, Y, dZ, perm_R, perm_P, Wt, g_R, g_P, q_R, q_P, H_save, dX, dg,
                        dg_first: int, dg_blocks: int, ws, ws_bytes: int, stream=None):
    _check(
        lib().poetx_linear_bwd_dx(
            ctypes.byref(dsc), T, _ptr(Y), _ptr(dZ), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _ptr(g_R), _ptr(g_P),
            _ptr(q_R), _ptr(q_P), _ptr(H_save), _ptr(dX), _ptr(dg), dg_first, dg_blocks, _ptr(ws), ws_bytes,
            _stream(stream),
        )
    )


def poetx_cnp_backward_batch_reuse(q, d, b: int, dtype: int, build_ws, build_ws_bytes: int, dg, dg_bytes: int, dq,
                                   stream=None):
    _check(lib().poetx_cnp_backward_batch_reuse(len(d), _ptr_array(q), _i32_array(d), b, dtype, _ptr(build_ws),
                                                build_ws_bytes, _ptr(dg), dg_bytes, _ptr_array(dq), _stream(stream)))


def poetx_linear_bwd_dx_sides(dsc: LayerDesc, T: int, Y, dZ, perm_R, perm_P, Wt, g_R, g_P, H_save, dX, ws,
                              ws_bytes: int, stream=None):
    """dX into `dX`; returns the two sides' block-gradient operands (R, P) as GradSide records."""
    sides = (GradSide * 2)()
    _check(
        lib().poetx_linear_bwd_dx_sides(
            ctypes.byref(dsc), T, _ptr(Y), _ptr(dZ), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _ptr(g_R), _ptr(g_P),
            _ptr(H_save), _ptr(dX), sides, _ptr(ws), ws_bytes, _stream(stream),
        )
    )
    return [sides[0], sides[1]]


def poetx_linear_fwd_group(calls, T: int, stream=None):
    """calls: list of dicts with the keyword arguments of poetx_linear_fwd (dsc, X, perm_R, perm_P, Wt, g_R, g_P,
    Y, H_save, ws, ws_bytes), marshalled into a host array of FwdCall records."""
    descs = [c["dsc"] for c in calls]  # kept alive through the call
    arr = (FwdCall * len(calls))(*[
        FwdCall(ctypes.pointer(dsc), _ptr(c["X"]), _ptr(c["perm_R"]), _ptr(c["perm_P"]), _ptr(c["Wt"]), _ptr(c["g_R"]),
                _ptr(c["g_P"]), _ptr(c["Y"]), _ptr(c["H_save"]), _ptr(c["ws"]), c["ws_bytes"])
        for c, dsc in zip(calls, descs)
    ])
    _check(lib().poetx_linear_fwd_group(len(calls), arr, T, _stream(stream)))


def poetx_linear_bwd_dx_group(calls, T: int, stream=None):
    """calls: list of dicts with the keyword arguments of poetx_linear_bwd_dx_sides (dsc, Y, dZ, perm_R, perm_P, Wt,
    g_R, g_P, H_save, dX, ws, ws_bytes); returns the block-gradient operands of every linear as pairs (R, P) of
    GradSide records."""
    descs = [c["dsc"] for c in calls]
    arr = (BwdCall * len(calls))(*[
        BwdCall(ctypes.pointer(dsc), _ptr(c["Y"]), _ptr(c["dZ"]), _ptr(c["perm_R"]), _ptr(c["perm_P"]), _ptr(c["Wt"]),
                _ptr(c["g_R"]), _ptr(c["g_P"]), _ptr(c["H_save"]), _ptr(c["dX"]), _ptr(c["ws"]), c["ws_bytes"])
        for c, dsc in zip(calls, descs)
    ])
    sides = (GradSide * (2 * len(calls)))()
    _check(lib().poetx_linear_bwd_dx_group(len(calls), arr, T, sides, _stream(stream)))
    return [[sides[2 * i], sides[2 * i + 1]] for i in range(len(calls))]


def poetx_block_grads_workspace_size(d, rows: int, b: int, dtype: int) -> int:
    return lib().poetx_block_grads_workspace_size(len(d), _i32_array(d), rows, b, dtype)


def poetx_block_grads_batch(sides, rows: int, b: int, dtype: int, dg, dg_bytes: int, ws, ws_bytes: int, stream=None):
    """sides: list of GradSide records (from poetx_linear_bwd_dx_sides), marshalled into a host array."""
    arr = (GradSide * len(sides))(*sides)
    _check(lib().poetx_block_grads_batch(len(sides), arr, rows, b, dtype, _ptr(dg), dg_bytes, _ptr(ws), ws_bytes,
                                         _stream(stream)))


def poetx_cnp_backward_batch(q, d, b: int, dtype: int, dg, dg_bytes: int, dq, stream=None):
    _check(lib().poetx_cnp_backward_batch(len(d), _ptr_array(q), _i32_array(d), b, dtype, _ptr(dg), dg_bytes,
                                          _ptr_array(dq), _stream(stream)))


# ------------------------------------------------- optimiser step on packed q ---
def poetx_adam_step_batch(q, dq, m1, m2, lr: float, beta1: float, beta2: float, eps: float, weight_decay: float,
                          t: int, lens=None, stream=None):
    """q, dq, m1, m2: per-side lists of fp32 device tensors; lens defaults to each q's numel()."""
    if lens is None:
        lens = [x.numel() for x in q]
    hp = AdamParams(lr, beta1, beta2, eps, weight_decay, t)
    _check(lib().poetx_adam_step_batch(len(lens), (ctypes.c_int64 * len(lens))(*lens), _ptr_array(q), _ptr_array(dq),
                                       _ptr_array(m1), _ptr_array(m2), ctypes.byref(hp), _stream(stream)))


# ------------------------------------------------------ orthogonalised updates ---
def ns_params(steps: int = 5, a: float = 3.4445, b: float = -4.7750, c: float = 2.0315, eps: float = 1e-7,
              rms: float = 0.2) -> NsParams:
    return NsParams(steps, a, b, c, eps, rms)


def muon_params(lr: float, beta: float = 0.95, weight_decay: float = 0.0, nesterov: bool = True, **ns) -> MuonParams:
    """ns: the keyword arguments of ns_params."""
    return MuonParams(lr, beta, weight_decay, int(nesterov), ns_params(**ns))


def poetx_muon_workspace_size(d, b: int) -> int:
    return lib().poetx_muon_workspace_size(len(d), _i32_array(d), b)


def poetx_muon_step_batch(q, dq, m, d, b: int, hp: MuonParams, ws, ws_bytes: int, stream=None):
    """q, dq, m, d: per-side lists (fp32 device tensors / ints), marshalled into host arrays."""
    _check(lib().poetx_muon_step_batch(len(d), _ptr_array(q), _ptr_array(dq), _ptr_array(m), _i32_array(d), b,
                                       ctypes.byref(hp), _ptr(ws), ws_bytes, _stream(stream)))


def poetx_orthogonalize_workspace_size(count: int, rows: int, cols: int, dtype: int) -> int:
    return lib().poetx_orthogonalize_workspace_size(count, rows, cols, dtype)


def poetx_orthogonalize(count: int, rows: int, cols: int, dtype: int, G, ld_g: int, stride_g: int, O, ld_o: int,
                        stride_o: int, hp: NsParams, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_orthogonalize(count, rows, cols, dtype, _ptr(G), ld_g, stride_g, _ptr(O), ld_o, stride_o,
                                     ctypes.byref(hp), _ptr(ws), ws_bytes, _stream(stream)))


# ------------------------------------------------------- norm of token rows ---
def norm_desc(d: int, kind: str, act: str, eps: float = 1e-5) -> NormDesc:
    return NormDesc(d, NORM_KINDS[kind], DTYPES[act], eps)


def poetx_norm_stats_bytes(dsc: NormDesc, T: int) -> int:
    return lib().poetx_norm_stats_bytes(ctypes.byref(dsc), T)


def poetx_norm_workspace_size(dsc: NormDesc, T: int) -> int:
    return lib().poetx_norm_workspace_size(ctypes.byref(dsc), T)


def poetx_norm_fwd(dsc: NormDesc, T: int, X, ldx: int, R, ldr: int, w, bias, S, lds: int, Y, ldy: int, stats,
                   stream=None):
    _check(lib().poetx_norm_fwd(ctypes.byref(dsc), T, _ptr(X), ldx, _ptr(R), ldr, _ptr(w), _ptr(bias), _ptr(S), lds,
                                _ptr(Y), ldy, _ptr(stats), _stream(stream)))


def poetx_norm_bwd(dsc: NormDesc, T: int, dY, lddy: int, S, lds: int, w, stats, dS, ldds: int, dX, lddx: int, dw,
                   dbias, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_norm_bwd(ctypes.byref(dsc), T, _ptr(dY), lddy, _ptr(S), lds, _ptr(w), _ptr(stats), _ptr(dS),
                                ldds, _ptr(dX), lddx, _ptr(dw), _ptr(dbias), _ptr(ws), ws_bytes, _stream(stream)))


# ---------------------------------------------------------- rotary positions ---
def rope_desc(head_dim: int, rot_dim: int, layout: str, act: str) -> RopeDesc:
    return RopeDesc(head_dim, rot_dim, ROPE_LAYOUTS[layout], DTYPES[act])


def rope_params(base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                low: float = 1.0, high: float = 4.0) -> RopeParams:
    return RopeParams(base, ROPE_SCALINGS[scaling], factor, original, low, high)


def poetx_rope_freqs(rot_dim: int, params: RopeParams):
    """(frequencies [rot_dim / 2] float64, amplitude) on the host."""
    import numpy as np

    out, amp = np.empty(max(rot_dim // 2, 1), dtype=np.float64), ctypes.c_float()
    _check(lib().poetx_rope_freqs(rot_dim, ctypes.byref(params), out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                  ctypes.byref(amp)))
    return out, amp.value


def poetx_rope(dsc: RopeDesc, T: int, pos, freqs, amplitude: float, inverse: bool, Xs, ldx, heads, Ys, ldy, stream=None):
    n = len(Xs)
    _check(lib().poetx_rope(ctypes.byref(dsc), T, _ptr(pos), _ptr(freqs), amplitude, int(inverse), n,
                            (ctypes.c_void_p * n)(*[_ptr(x) for x in Xs]), (ctypes.c_int64 * n)(*ldx),
                            (ctypes.c_int32 * n)(*heads), (ctypes.c_void_p * n)(*[_ptr(y) for y in Ys]),
                            (ctypes.c_int64 * n)(*ldy), _stream(stream)))


# ------------------------------------------------ attention of packed sequences ---
def attn_desc(heads: int, kv_heads: int, head_dim: int, act: str, causal: bool = True, window: int = 0,
              scale: Optional[float] = None) -> AttnDesc:
    """scale: 1 / sqrt(head_dim) where it is None."""
    if scale is None:
        scale = head_dim**-0.5
    return AttnDesc(heads, kv_heads, head_dim, DTYPES[act], int(causal), window, scale)


def poetx_attn_workspace_size(dsc: AttnDesc, batch: int, Tq: int, Tk: int, op: int) -> int:
    return lib().poetx_attn_workspace_size(ctypes.byref(dsc), batch, Tq, Tk, op)


def poetx_attn_fwd(dsc: AttnDesc, batch: int, Tq: int, Tk: int, cu_q, cu_k, Q, ldq: int, K, ldk: int, V, ldv: int, O,
                   ldo: int, lse, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_attn_fwd(ctypes.byref(dsc), batch, Tq, Tk, _ptr(cu_q), _ptr(cu_k), _ptr(Q), ldq, _ptr(K), ldk,
                                _ptr(V), ldv, _ptr(O), ldo, _ptr(lse), _ptr(ws), ws_bytes, _stream(stream)))


def poetx_attn_bwd(dsc: AttnDesc, batch: int, Tq: int, Tk: int, cu_q, cu_k, dO, lddo: int, Q, ldq: int, K, ldk: int, V,
                   ldv: int, O, ldo: int, lse, dQ, lddq: int, dK, lddk: int, dV, lddv: int, ws, ws_bytes: int,
                   stream=None):
    _check(lib().poetx_attn_bwd(ctypes.byref(dsc), batch, Tq, Tk, _ptr(cu_q), _ptr(cu_k), _ptr(dO), lddo, _ptr(Q), ldq,
                                _ptr(K), ldk, _ptr(V), ldv, _ptr(O), ldo, _ptr(lse), _ptr(dQ), lddq, _ptr(dK), lddk,
                                _ptr(dV), lddv, _ptr(ws), ws_bytes, _stream(stream)))


# ---------------------------------------------- log probabilities of given tokens ---
def logp_desc(vocab: int, act: str, top: int = 0, scale: float = 1.0) -> LogpDesc:
    return LogpDesc(vocab, DTYPES[act], top, scale)


def poetx_logp_workspace_size(dsc: LogpDesc, T: int) -> int:
    return lib().poetx_logp_workspace_size(ctypes.byref(dsc), T)


def poetx_logp_fwd(dsc: LogpDesc, T: int, X, ldx: int, target, logp, lse, entropy, top_ids, top_logp, ws, ws_bytes: int,
                   stream=None):
    _check(lib().poetx_logp_fwd(ctypes.byref(dsc), T, _ptr(X), ldx, _ptr(target), _ptr(logp), _ptr(lse), _ptr(entropy),
                                _ptr(top_ids), _ptr(top_logp), _ptr(ws), ws_bytes, _stream(stream)))


def poetx_logp_bwd(dsc: LogpDesc, T: int, X, ldx: int, target, lse, entropy, dlogp, dentropy, dX, lddx: int,
                   stream=None):
    _check(lib().poetx_logp_bwd(ctypes.byref(dsc), T, _ptr(X), ldx, _ptr(target), _ptr(lse), _ptr(entropy), _ptr(dlogp),
                                _ptr(dentropy), _ptr(dX), lddx, _stream(stream)))


# ------------------------------------------------------------ one SPO factor ---
def spo_desc(d: int, b: int, kind: str, act: str) -> SpoDesc:
    return SpoDesc(d, b, SPO_KINDS[kind], DTYPES[act])


def poetx_spo_saved_bytes(dsc: SpoDesc, T: int) -> int:
    return lib().poetx_spo_saved_bytes(ctypes.byref(dsc), T)


def poetx_spo_workspace_size(dsc: SpoDesc, T: int, op: int) -> int:
    return lib().poetx_spo_workspace_size(ctypes.byref(dsc), T, op)


def poetx_spo_fwd(dsc: SpoDesc, T: int, X, idx, G, Y, saved, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_spo_fwd(ctypes.byref(dsc), T, _ptr(X), _ptr(idx), _ptr(G), _ptr(Y), _ptr(saved), _ptr(ws),
                               ws_bytes, _stream(stream)))


def poetx_spo_bwd(dsc: SpoDesc, T: int, dY, idx, G, q, saved, dX, dq, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_spo_bwd(ctypes.byref(dsc), T, _ptr(dY), _ptr(idx), _ptr(G), _ptr(q), _ptr(saved), _ptr(dX),
                               _ptr(dq), _ptr(ws), ws_bytes, _stream(stream)))


# --------------------------------------------------- weight-centric baseline ---
def poetx_wc_state_bytes(dsc: LayerDesc, T: int) -> int:
    return lib().poetx_wc_state_bytes(ctypes.byref(dsc), T)


def poetx_wc_workspace_size(dsc: LayerDesc, T: int, op: int) -> int:
    return lib().poetx_wc_workspace_size(ctypes.byref(dsc), T, op)


def poetx_wc_fwd(dsc: LayerDesc, T: int, X, perm_R, perm_P, Wt, g_R, g_P, Y, state, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_wc_fwd(ctypes.byref(dsc), T, _ptr(X), _ptr(perm_R), _ptr(perm_P), _ptr(Wt), _ptr(g_R), _ptr(g_P),
                              _ptr(Y), _ptr(state), _ptr(ws), ws_bytes, _stream(stream)))


def poetx_wc_bwd(dsc: LayerDesc, T: int, dZ, perm_R, perm_P, g_R, g_P, q_R, q_P, state, dX, dq_R, dq_P, ws,
                 ws_bytes: int, stream=None):
    _check(lib().poetx_wc_bwd(ctypes.byref(dsc), T, _ptr(dZ), _ptr(perm_R), _ptr(perm_P), _ptr(g_R), _ptr(g_P),
                              _ptr(q_R), _ptr(q_P), _ptr(state), _ptr(dX), _ptr(dq_R), _ptr(dq_P), _ptr(ws), ws_bytes,
                              _stream(stream)))


# ---------------------------------------- merging a chain's outer factors ---
def poetx_fold_workspace_size(dsc: LayerDesc, side: int, f: SpoDesc) -> int:
    return lib().poetx_fold_workspace_size(ctypes.byref(dsc), side, ctypes.byref(f))


def poetx_fold_factor(dsc: LayerDesc, side: int, f: SpoDesc, idx, G, perm, W, ldw: int, ws, ws_bytes: int,
                      stream=None):
    _check(lib().poetx_fold_factor(ctypes.byref(dsc), side, ctypes.byref(f), _ptr(idx), _ptr(G), _ptr(perm), _ptr(W),
                                   ldw, _ptr(ws), ws_bytes, _stream(stream)))


def poetx_store_workspace_size(dsc: LayerDesc) -> int:
    return lib().poetx_store_workspace_size(ctypes.byref(dsc))


def poetx_store_weight(dsc: LayerDesc, W, ldw: int, Wt, ws, ws_bytes: int, stream=None):
    _check(lib().poetx_store_weight(ctypes.byref(dsc), _ptr(W), ldw, _ptr(Wt), _ptr(ws), ws_bytes, _stream(stream)))
