"""Python binding of liborbitquant: argument marshalling only.

Every function has the name of the C entry point it calls
(include/orbitquant.h).  Torch tensors provide device memory and the current
stream; all compute runs in the library's CUDA kernels.  There is no fallback:
if the library is missing or no GPU is present the calls raise.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liborbitquant.so")

OQ_OK = 0
OQ_DTYPE_F32 = 0
OQ_DTYPE_BF16 = 1
OQ_FLAG_SIGNS = 1
OQ_FLAG_GAUSSIAN_MARGINAL = 2
OQ_FLAG_WEIGHT_ONLY_INT4 = 4
OQ_FLAG_FP8_CONTRACTION = 8
OQ_FLAG_MICROSCALED = 16
OQ_QK_INTERLEAVED = 1
OQ_QK_NO_NORM = 2
OQ_ATTN_CAUSAL = 1
OQ_KV4_PAGE = 128      # tokens of a page of the 4-bit cache
# oq_linear_fused decodes the weight codes once per call from this many tokens
# on (bf16 x, d_out % 256 == 0, a workspace of oq_linear_fused_workspace_size)
W16_MIN_T = 1024

# every symbol include/orbitquant.h declares
EXPORTS = (
    "oq_codebook_build", "oq_rotation_build", "oq_layer_create", "oq_layer_destroy", "oq_layer_get_info", "oq_layer_get_perm",
    "oq_rotate_quantize", "oq_weight_prepare", "oq_weight_save", "oq_weight_load", "oq_linear",
    "oq_linear_fused_workspace_size",
    "oq_linear_fused", "oq_linear_fused_decoded_workspace_size", "oq_linear_fused_decoded",
    "oq_rotate_quantize_levels", "oq_linear_levels", "oq_weight_levels", "oq_linear_decoded",
    "oq_linear_fused_static", "oq_linear_fused_host_workspace_size", "oq_linear_fused_host",
    "oq_mx_codes_size", "oq_mx_scales_size", "oq_mx_quantize", "oq_mx_dequantize", "oq_rms_norm_mx", "oq_linear_mx",
    "oq_qk_norm_rope", "oq_kv4_create", "oq_kv4_destroy", "oq_kv4_cache_size", "oq_kv4_append", "oq_kv4_read",
    "oq_kv4_attention_workspace_size", "oq_kv4_attention", "oq_kv4_poll_error", "oq_w4g_prepare", "oq_linear_w4g",
    "oq_poll_error", "oq_check_wait_timeout", "oq_last_error", "oq_status_string",
)


class OrbitQuantError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


class LibraryMissing(OrbitQuantError):
    pass


class CodebookC(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("bits", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("iterations", ctypes.c_int32), ("levels", ctypes.c_double * 256),
                ("thresholds", ctypes.c_double * 255), ("mse", ctypes.c_double)]


class LayerInfoC(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("h", ctypes.c_int32),
                ("k", ctypes.c_int32), ("a_bits", ctypes.c_int32), ("w_bits", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("a_words_per_row", ctypes.c_int64), ("w_words_per_row", ctypes.c_int64),
                ("a_scale", ctypes.c_double), ("w_scale", ctypes.c_double)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load liborbitquant.so (raises LibraryMissing if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise LibraryMissing(-1, "load_library",
                             f"{path} not found; build it with `python -m quantized_linear_token_b200.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
    sigs = {
        "oq_codebook_build": (i32, [i32, i32, i32, ctypes.POINTER(CodebookC)]),
        "oq_rotation_build": (i32, [i32, u64, i32, vp, vp]),
        "oq_layer_create": (i32, [i32, i32, u64, i32, i32, i32, ctypes.POINTER(vp)]),
        "oq_layer_destroy": (None, [vp]),
        "oq_layer_get_info": (i32, [vp, ctypes.POINTER(LayerInfoC)]),
        "oq_layer_get_perm": (i32, [vp, vp]),
        "oq_rotate_quantize": (i32, [vp, vp, i32, i64, vp, vp, vp]),
        "oq_weight_prepare": (i32, [vp, vp, i32, vp, vp, vp]),
        "oq_linear": (i32, [vp, vp, vp, i64, vp, vp, vp, i32, vp]),
        "oq_linear_fused_workspace_size": (sz, [vp, i64]),
        "oq_linear_fused": (i32, [vp, vp, i32, i64, vp, vp, vp, i32, vp, sz, vp]),
        "oq_rotate_quantize_levels": (i32, [vp, vp, i32, i64, vp, vp, vp]),
        "oq_linear_levels": (i32, [vp, vp, vp, i64, vp, vp, vp, i32, vp]),
        "oq_weight_levels": (i32, [vp, vp, vp, vp]),
        "oq_linear_fused_host_workspace_size": (ctypes.c_size_t, [vp, i32, i64]),
        "oq_linear_fused_host": (i32, [vp, vp, i32, i64, vp, vp, vp, i32, vp, ctypes.c_size_t, vp]),
        "oq_linear_decoded": (i32, [vp, vp, vp, i64, vp, vp, vp, i32, vp]),
        "oq_linear_fused_decoded_workspace_size": (sz, [vp, i64]),
        "oq_linear_fused_decoded": (i32, [vp, vp, i32, i64, vp, vp, vp, i32, vp, sz, vp]),
        "oq_linear_fused_static": (i32, [vp, vp, i32, i64, vp, vp, vp, vp]),
        "oq_weight_save": (i32, [vp, vp, vp, ctypes.c_char_p]),
        "oq_weight_load": (i32, [vp, ctypes.c_char_p, vp, vp]),
        "oq_mx_codes_size": (sz, [i64, i32, i32]),
        "oq_mx_scales_size": (sz, [i64, i32]),
        "oq_mx_quantize": (i32, [vp, i32, i64, i32, i32, vp, vp, vp]),
        "oq_mx_dequantize": (i32, [vp, vp, i64, i32, i32, vp, i32, vp]),
        "oq_rms_norm_mx": (i32, [vp, vp, i32, vp, i32, ctypes.c_float, i64, i32, i32, vp, vp, vp, vp]),
        "oq_linear_mx": (i32, [vp, vp, vp, i64, vp, vp, vp, i32, vp]),
        "oq_qk_norm_rope": (i32, [vp, i64, i32, vp, i64, i32, i32, i64, i32, vp, vp, i32, ctypes.c_float, vp, i64, i32, vp,
                                  i32, vp, i64, vp, i64, vp]),
        "oq_kv4_create": (i32, [i32, i32, i32, ctypes.POINTER(vp)]),
        "oq_kv4_destroy": (None, [vp]),
        "oq_kv4_cache_size": (sz, [vp, i64]),
        "oq_kv4_append": (i32, [vp, vp, i64, vp, i64, vp, i64, i32, i64, vp, vp, i32, ctypes.c_float, vp, i64, i32, vp, i32,
                                vp, vp, i64, vp, i32, vp, vp, i32, vp]),
        "oq_kv4_read": (i32, [vp, vp, i64, vp, i32, vp, vp, i32, i64, vp, vp, i32, vp]),
        "oq_kv4_attention_workspace_size": (sz, [vp, i64, i32, i32, i32]),
        "oq_kv4_attention": (i32, [vp, vp, i64, i64, vp, i64, vp, i32, vp, vp, i32, i32, i32, ctypes.c_float, i32, i32, vp,
                                   vp, sz, vp]),
        "oq_kv4_poll_error": (i32, [vp]),
        "oq_w4g_prepare": (i32, [vp, i32, i32, i32, i32, vp, vp, vp, vp]),
        "oq_linear_w4g": (i32, [vp, i32, i64, i32, i32, i32, vp, vp, vp, vp, i32, vp]),
        "oq_poll_error": (i32, [vp]),
        "oq_check_wait_timeout": (i32, [vp, ctypes.c_uint32, vp]),
        "oq_last_error": (ctypes.c_char_p, []),
        "oq_status_string": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status: int, where: str):
    if status != OQ_OK:
        L = load_library()
        raise OrbitQuantError(status, where, L.oq_last_error().decode() or L.oq_status_string(status).decode())


# ------------------------------------------------------------------ host calls
def oq_codebook_build(d: int, bits: int, flags: int = 0) -> dict:
    """Lloyd-Max codebook C_{d,bits} as designed by the library (host)."""
    cb = CodebookC()
    _check(load_library().oq_codebook_build(d, bits, flags, ctypes.byref(cb)), "oq_codebook_build")
    L = 1 << bits
    return {"d": cb.d, "bits": cb.bits, "flags": cb.flags, "iterations": cb.iterations,
            "levels": np.array(cb.levels[:L]), "thresholds": np.array(cb.thresholds[:L - 1]), "mse": cb.mse}


def oq_rotation_build(d: int, seed: int, flags: int = 0):
    """(perm [d] uint32, signs [d] int8 or None) of the seeded rotation (host)."""
    perm = np.empty(d, dtype=np.uint32)
    signs = np.empty(d, dtype=np.int8) if flags & OQ_FLAG_SIGNS else None
    _check(load_library().oq_rotation_build(d, seed, flags, perm.ctypes.data,
                                            None if signs is None else signs.ctypes.data), "oq_rotation_build")
    return perm, signs


class Layer:
    """Owns an oq_layer* (the shared rotation, codebooks and device tables)."""

    def __init__(self, handle: int, lib):
        self._h = ctypes.c_void_p(handle)
        self._lib = lib
        info = LayerInfoC()
        _check(lib.oq_layer_get_info(self._h, ctypes.byref(info)), "oq_layer_get_info")
        self.d_in, self.d_out, self.h, self.k = info.d_in, info.d_out, info.h, info.k
        self.a_bits, self.w_bits, self.flags, self.seed = info.a_bits, info.w_bits, info.flags, info.seed
        self.a_words_per_row, self.w_words_per_row = info.a_words_per_row, info.w_words_per_row
        self.a_scale, self.w_scale = info.a_scale, info.w_scale

    @property
    def handle(self):
        return self._h

    def perm(self) -> np.ndarray:
        out = np.empty(self.d_in, dtype=np.uint32)
        _check(self._lib.oq_layer_get_perm(self._h, out.ctypes.data), "oq_layer_get_perm")
        return out

    def close(self):
        if self._h:
            self._lib.oq_layer_destroy(self._h)
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def oq_layer_create(d_in: int, d_out: int, seed: int, a_bits: int, w_bits: int, flags: int = 0) -> Layer:
    L = load_library()
    h = ctypes.c_void_p()
    _check(L.oq_layer_create(d_in, d_out, seed, a_bits, w_bits, flags, ctypes.byref(h)), "oq_layer_create")
    return Layer(h.value, L)


# ------------------------------------------------------------------ device calls
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return OQ_DTYPE_BF16
    if t.dtype == torch.float32:
        return OQ_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


def _dev(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def oq_rotate_quantize(layer: Layer, x, codes=None, s=None):
    """x [T, d_in] (bf16/fp32, CUDA) -> (codes [T, d_in*a_bits/32] int32 view of uint32, s [T] fp32)."""
    torch = _torch()
    T = x.shape[0]
    if x.dim() != 2 or x.shape[1] != layer.d_in:
        raise ValueError("x must be [T, d_in]")
    if codes is None:
        codes = torch.empty((T, layer.a_words_per_row), dtype=torch.int32, device=x.device)
    if s is None:
        s = torch.empty((T,), dtype=torch.float32, device=x.device)
    _check(load_library().oq_rotate_quantize(layer.handle, _dev(x, "x"), _dtype_code(x), T, _dev(codes, "codes"),
                                             _dev(s, "s"), _stream(x)), "oq_rotate_quantize")
    return codes, s


def oq_weight_prepare(layer: Layer, W, Wcodes=None, r=None):
    """W [d_out, d_in] (fp32/bf16, CUDA) -> (Wcodes [d_out, d_in*w_bits/32] int32, r [d_out] fp32)."""
    torch = _torch()
    if W.dim() != 2 or tuple(W.shape) != (layer.d_out, layer.d_in):
        raise ValueError("W must be [d_out, d_in]")
    if Wcodes is None:
        Wcodes = torch.empty((layer.d_out, layer.w_words_per_row), dtype=torch.int32, device=W.device)
    if r is None:
        r = torch.empty((layer.d_out,), dtype=torch.float32, device=W.device)
    _check(load_library().oq_weight_prepare(layer.handle, _dev(W, "W"), _dtype_code(W), _dev(Wcodes, "Wcodes"),
                                            _dev(r, "r"), _stream(W)), "oq_weight_prepare")
    return Wcodes, r


def _y_out(y, T: int, d_out: int, y_dtype, device):
    """The output tensor (given, or new of y_dtype: torch.float32 or
    torch.bfloat16) and its C dtype code."""
    torch = _torch()
    if y is None:
        y = torch.empty((T, d_out), dtype=torch.float32 if y_dtype is None else y_dtype, device=device)
    if y.dtype == torch.float32:
        return y, OQ_DTYPE_F32
    if y.dtype == torch.bfloat16:
        return y, OQ_DTYPE_BF16
    raise ValueError("y must be float32 or bfloat16")


def oq_linear(layer: Layer, codes, s, Wcodes, r, y=None, y_dtype=None):
    """(codes, s, Wcodes, r) -> y [T, d_out] fp32 (or bf16)."""
    T = codes.shape[0]
    y, ycode = _y_out(y, T, layer.d_out, y_dtype, codes.device)
    _check(load_library().oq_linear(layer.handle, _dev(codes, "codes"), _dev(s, "s"), T, _dev(Wcodes, "Wcodes"),
                                    _dev(r, "r"), _dev(y, "y"), ycode, _stream(codes)), "oq_linear")
    return y


def oq_linear_fused_workspace_size(layer: Layer, T: int) -> int:
    return int(load_library().oq_linear_fused_workspace_size(layer.handle, T))


def oq_linear_fused(layer: Layer, x, Wcodes, r, y=None, workspace=None, y_dtype=None):
    """x [T, d_in] -> y [T, d_out] fp32 (or bf16) in one call."""
    torch = _torch()
    T = x.shape[0]
    y, ycode = _y_out(y, T, layer.d_out, y_dtype, x.device)
    need = oq_linear_fused_workspace_size(layer, T)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=x.device)
    _check(load_library().oq_linear_fused(layer.handle, _dev(x, "x"), _dtype_code(x), T, _dev(Wcodes, "Wcodes"),
                                          _dev(r, "r"), _dev(y, "y"), ycode, _dev(workspace, "workspace"),
                                          workspace.numel() * workspace.element_size(), _stream(x)),
           "oq_linear_fused")
    return y


def oq_rotate_quantize_levels(layer: Layer, x, a16=None, s=None):
    """x [T, d_in] bf16 (CUDA) -> (a16 [T, d_in] fp16 levels of the codes, s [T] fp32):
    the first stage of the fused call's fp16 route."""
    torch = _torch()
    T = x.shape[0]
    if a16 is None:
        a16 = torch.empty((T, layer.d_in), dtype=torch.float16, device=x.device)
    if s is None:
        s = torch.empty((T,), dtype=torch.float32, device=x.device)
    _check(load_library().oq_rotate_quantize_levels(layer.handle, _dev(x, "x"), _dtype_code(x), T, _dev(a16, "a16"),
                                                    _dev(s, "s"), _stream(x)), "oq_rotate_quantize_levels")
    return a16, s


def oq_linear_levels(layer: Layer, a16, s, Wcodes, r, y=None, y_dtype=None):
    """(a16 fp16 levels, s, Wcodes, r) -> y [T, d_out] fp32 (or bf16): the
    second stage of the fused call's fp16 route."""
    T = a16.shape[0]
    y, ycode = _y_out(y, T, layer.d_out, y_dtype, a16.device)
    _check(load_library().oq_linear_levels(layer.handle, _dev(a16, "a16"), _dev(s, "s"), T, _dev(Wcodes, "Wcodes"),
                                           _dev(r, "r"), _dev(y, "y"), ycode, _stream(a16)), "oq_linear_levels")
    return y


def oq_weight_levels(layer: Layer, Wcodes, w16=None):
    """Wcodes [d_out, d_in*w_bits/32] -> w16 [d_out, d_in] fp16 levels of the
    weight codes (decoded once; the large-batch route's B operand)."""
    torch = _torch()
    if w16 is None:
        w16 = torch.empty((layer.d_out, layer.d_in), dtype=torch.float16, device=Wcodes.device)
    _check(load_library().oq_weight_levels(layer.handle, _dev(Wcodes, "Wcodes"), _dev(w16, "w16"), _stream(Wcodes)),
           "oq_weight_levels")
    return w16


def oq_linear_decoded(layer: Layer, a16, s, w16, r, y=None, y_dtype=None):
    """(a16, s, w16, r) -> y [T, d_out] fp32 (or bf16): the contraction of two
    fp16 level operands, both read by TMA."""
    T = a16.shape[0]
    y, ycode = _y_out(y, T, layer.d_out, y_dtype, a16.device)
    _check(load_library().oq_linear_decoded(layer.handle, _dev(a16, "a16"), _dev(s, "s"), T, _dev(w16, "w16"),
                                            _dev(r, "r"), _dev(y, "y"), ycode, _stream(a16)), "oq_linear_decoded")
    return y


def oq_linear_fused_decoded_workspace_size(layer: Layer, T: int) -> int:
    return int(load_library().oq_linear_fused_decoded_workspace_size(layer.handle, T))


def oq_linear_fused_decoded(layer: Layer, x, w16, r, y=None, workspace=None, y_dtype=None):
    """x [T, d_in] bf16 and the weights' fp16 levels w16 -> y [T, d_out]: the
    fused call's large-batch route after its weight decode (one kernel
    rotating, quantizing and contracting where the block size allows)."""
    torch = _torch()
    T = x.shape[0]
    y, ycode = _y_out(y, T, layer.d_out, y_dtype, x.device)
    if workspace is None:
        workspace = torch.empty((max(oq_linear_fused_decoded_workspace_size(layer, T), 1),), dtype=torch.uint8,
                                device=x.device)
    _check(load_library().oq_linear_fused_decoded(layer.handle, _dev(x, "x"), _dtype_code(x), T, _dev(w16, "w16"),
                                                  _dev(r, "r"), _dev(y, "y"), ycode, _dev(workspace, "workspace"),
                                                  workspace.numel() * workspace.element_size(), _stream(x)),
           "oq_linear_fused_decoded")
    return y


def oq_linear_fused_host_workspace_size(layer: Layer, x_dtype: int, T: int) -> int:
    return int(load_library().oq_linear_fused_host_workspace_size(layer.handle, x_dtype, T))


def _host(t, name: str):
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def oq_linear_fused_host(layer: Layer, x_host, Wcodes, r, y_host=None, workspace=None, y_dtype=None):
    """x_host [T, d_in] bf16/fp32 in host memory (pinned for overlap) -> y_host
    [T, d_out] fp32 in host memory: copies in, the fused call and copies out,
    overlapped chunk by chunk, queued on the current stream of Wcodes' device.
    Synchronise that stream before reading y_host."""
    torch = _torch()
    T = x_host.shape[0]
    if x_host.dim() != 2 or x_host.shape[1] != layer.d_in:
        raise ValueError("x_host must be [T, d_in]")
    if y_host is None:
        y_host = torch.empty((T, layer.d_out), dtype=torch.float32 if y_dtype is None else y_dtype, pin_memory=True)
    if y_host.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("y_host must be float32 or bfloat16")
    ycode = OQ_DTYPE_F32 if y_host.dtype == torch.float32 else OQ_DTYPE_BF16
    code = _dtype_code(x_host)
    need = oq_linear_fused_host_workspace_size(layer, code, T)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=Wcodes.device)
    _check(load_library().oq_linear_fused_host(layer.handle, _host(x_host, "x_host"), code, T,
                                               _dev(Wcodes, "Wcodes"), _dev(r, "r"), _host(y_host, "y_host"), ycode,
                                               _dev(workspace, "workspace"),
                                               workspace.numel() * workspace.element_size(), _stream(Wcodes)),
           "oq_linear_fused_host")
    return y_host


def oq_linear_fused_static(layer: Layer, x, Wcodes, r, y=None):
    """x [T, d_in] -> y [T, d_out] fp32 without any device allocation by the
    library: its scratch is a fixed array the library reserves per GPU (see
    include/orbitquant.h).  Calls that overlap on the GPU race on it."""
    torch = _torch()
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, layer.d_out), dtype=torch.float32, device=x.device)
    _check(load_library().oq_linear_fused_static(layer.handle, _dev(x, "x"), _dtype_code(x), T,
                                                 _dev(Wcodes, "Wcodes"), _dev(r, "r"), _dev(y, "y"), _stream(x)),
           "oq_linear_fused_static")
    return y


def oq_weight_save(layer: Layer, Wcodes, r, path: str) -> None:
    """Write prepared weights (device Wcodes, r from oq_weight_prepare) to a file."""
    _check(load_library().oq_weight_save(layer.handle, _dev(Wcodes, "Wcodes"), _dev(r, "r"),
                                         os.fsencode(path)), "oq_weight_save")


def oq_weight_load(layer: Layer, path: str, Wcodes=None, r=None):
    """Read prepared weights saved for a layer with the same settings ->
    (Wcodes, r) on the current CUDA device."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device())
    if Wcodes is None:
        Wcodes = torch.empty((layer.d_out, layer.w_words_per_row), dtype=torch.int32, device=dev)
    if r is None:
        r = torch.empty((layer.d_out,), dtype=torch.float32, device=dev)
    _check(load_library().oq_weight_load(layer.handle, os.fsencode(path), _dev(Wcodes, "Wcodes"), _dev(r, "r")),
           "oq_weight_load")
    return Wcodes, r


# ------------------------------------------------------------------ microscaled operators
def oq_mx_codes_size(rows: int, d: int, bits: int) -> int:
    return int(load_library().oq_mx_codes_size(rows, d, bits))


def oq_mx_scales_size(rows: int, d: int) -> int:
    return int(load_library().oq_mx_scales_size(rows, d))


_raw = None   # (current device, raw current stream of a device, uint8, dtype codes), on first use


def _raw_calls():
    global _raw
    torch = _torch()
    _raw = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream, torch.uint8,
            {torch.float32: OQ_DTYPE_F32, torch.bfloat16: OQ_DTYPE_BF16})
    return _raw


def _launch(name: str, device, *args):
    """Call an entry point with `device` current and its current stream as the
    last argument.  Small calls are bound by the host, so this and the checks
    below spend as little as they can."""
    get_device, get_stream, _, _ = _raw or _raw_calls()
    fn = getattr(_lib or load_library(), name)
    i = device.index
    if get_device() == i:
        status = fn(*args, get_stream(i))
    else:
        with _torch().cuda.device(device):
            status = fn(*args, get_stream(i))
    if status:
        _check(status, name)


def _mx_ptr(t, shape, device, name: str) -> int:
    """The address of a contiguous uint8 tensor of this shape on `device`."""
    if t.dtype is not (_raw or _raw_calls())[2] or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous uint8 {list(shape)} on {device}")
    return t.data_ptr()


def _mx_dtype(t) -> int:
    code = (_raw or _raw_calls())[3].get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")
    return code


def _mx_input(x, name: str, bits: int) -> int:
    """The address of a [rows, d] operand to quantize."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    d = x.shape[1]
    if (bits != 4 and bits != 8) or d == 0 or d % 32:
        raise ValueError(f"bits must be 4 or 8 and {name}'s width a positive multiple of 32")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return x.data_ptr()


def _mx_shapes(rows: int, d: int, bits: int):
    """Shapes of the codes and the scale tiles of a [rows, d] operand."""
    ct = (d + 127) // 128
    return (rows, ct * 16 * bits), ((rows + 127) // 128, ct, 32, 4, 4)


def _mx_outputs(codes, scales, rows: int, d: int, bits: int, device):
    """Codes and scales to write: new ones, or the given ones checked; and their addresses."""
    torch = _torch()
    if device.type != "cuda":
        raise ValueError("the operands must be CUDA tensors")
    cs, ss = _mx_shapes(rows, d, bits)
    if codes is None:
        # (empty_strided takes two thirds of the time of empty)
        codes = torch.empty_strided(cs, (cs[1], 1), dtype=torch.uint8, device=device)
        pc = codes.data_ptr()
    else:
        pc = _mx_ptr(codes, cs, device, "codes")
    if scales is None:
        scales = torch.empty_strided(ss, (512 * ss[1], 512, 16, 4, 1), dtype=torch.uint8, device=device)
        ps = scales.data_ptr()
    else:
        ps = _mx_ptr(scales, ss, device, "scales")
    return codes, scales, pc, ps


def _mx_rows(t, shape, dtype, device, name: str) -> int:
    """The address of a contiguous tensor of this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {device}")
    return t.data_ptr()


def oq_mx_quantize(x, bits: int, codes=None, scales=None):
    """x [rows, d] (bf16/fp32, CUDA) -> (codes [rows, row bytes] uint8, scales
    [row tiles, column tiles, 32, 4, 4] uint8): microscaled e2m1 (bits = 4) or
    e4m3 (bits = 8) elements, one E8M0 scale per 32 (include/orbitquant.h)."""
    px, dt, device = _mx_input(x, "x", bits), _mx_dtype(x), x.device
    rows, d = x.shape
    codes, scales, pc, ps = _mx_outputs(codes, scales, rows, d, bits, device)
    _launch("oq_mx_quantize", device, px, dt, rows, d, bits, pc, ps)
    return codes, scales


def oq_mx_dequantize(codes, scales, d: int, bits: int, dtype=None, x=None):
    """Codes and scales of a [rows, d] operand -> its values [rows, d] (fp32 by
    default, or bf16)."""
    torch = _torch()
    if codes.dim() != 2 or scales is None or bits not in (4, 8) or d <= 0 or d % 32:
        raise ValueError("codes must be a matrix with its scales, bits 4 or 8 and d a positive multiple of 32")
    rows, device = codes.shape[0], codes.device
    _, _, pc, ps = _mx_outputs(codes, scales, rows, d, bits, device)
    if x is None:
        x = torch.empty_strided((rows, d), (d, 1), dtype=torch.float32 if dtype is None else dtype, device=device)
        px = x.data_ptr()
    else:
        px = _mx_rows(x, (rows, d), x.dtype if dtype is None else dtype, device, "x")
    _launch("oq_mx_dequantize", device, pc, ps, rows, d, bits, px, _mx_dtype(x))
    return x


def oq_rms_norm_mx(x, gain=None, residual=None, eps: float = 1e-6, bits: int = 8, residual_out=None, codes=None,
                   scales=None):
    """h = x + residual, its root-mean-square norm times gain, quantized: x,
    residual [rows, d] (bf16/fp32, CUDA), gain [d] -> (codes, scales, h rounded
    to x's type, or None without a residual).  residual_out may be x or
    residual itself."""
    torch = _torch()
    px, dt = _mx_input(x, "x", bits), _mx_dtype(x)
    rows, d = shape = x.shape
    dtype, device = x.dtype, x.device
    pr = po = pg = None
    gdt = OQ_DTYPE_F32
    if residual is not None:
        pr = _mx_rows(residual, shape, dtype, device, "residual")
        if residual_out is None:
            residual_out = torch.empty_like(x)
            po = residual_out.data_ptr()
        else:
            po = _mx_rows(residual_out, shape, dtype, device, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if gain is not None:
        gdt, pg = _mx_dtype(gain), _mx_rows(gain, (d,), gain.dtype, device, "gain")
    codes, scales, pc, ps = _mx_outputs(codes, scales, rows, d, bits, device)
    _launch("oq_rms_norm_mx", device, px, pr, dt, pg, gdt, eps, rows, d, bits, po, pc, ps)
    return codes, scales, residual_out


def oq_linear_mx(layer: Layer, codes, scales, Wcodes, Wscales, y=None, y_dtype=None):
    """Microscaled activations (codes, scales of layer.a_bits) times 4-bit
    microscaled weights -> y [T, d_out] fp32 (or bf16), on a layer created with
    OQ_FLAG_MICROSCALED."""
    if not layer.flags & OQ_FLAG_MICROSCALED:
        raise ValueError("the layer was not created with OQ_FLAG_MICROSCALED")
    if codes.dim() != 2 or not codes.is_cuda:
        raise ValueError("codes must be a CUDA matrix")
    T, device, n = codes.shape[0], codes.device, layer.d_out
    cs, ss = _mx_shapes(T, layer.d_in, layer.a_bits)
    ws, wt = _mx_shapes(n, layer.d_in, 4)
    pointers = (_mx_ptr(codes, cs, device, "codes"), _mx_ptr(scales, ss, device, "scales"), T,
                _mx_ptr(Wcodes, ws, device, "Wcodes"), _mx_ptr(Wscales, wt, device, "Wscales"))
    if y is None:
        torch = _torch()
        y = torch.empty_strided((T, n), (n, 1), dtype=torch.float32 if y_dtype is None else y_dtype, device=device)
        py = y.data_ptr()
    else:
        py = _mx_rows(y, (T, n), y.dtype if y_dtype is None else y_dtype, device, "y")
    ycode = _mx_dtype(y)
    _launch("oq_linear_mx", device, layer.handle, *pointers, py, ycode)
    return y


# ------------------------------------------------------------------ operators around attention
def _heads(t, heads, D: int, device, name: str):
    """(address, token stride) of a [T, heads, D] tensor whose tokens' heads are contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads) or t.device != device:
        raise ValueError(f"{name} must be [T, {'heads' if heads is None else heads}, {D}] on {device}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1 or s1 != D and shape[1] > 1) and t.numel():
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), s0 if shape[0] > 1 else shape[1] * D


def _ints(t, shape, device, name: str) -> int:
    """The address of a contiguous int32 tensor of this shape on `device`."""
    if t.dtype is not _int32() or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)} on {device}")
    return t.data_ptr()


_i32 = None


def _int32():
    global _i32
    if _i32 is None:
        _i32 = _torch().int32
    return _i32


def _new_heads(T: int, heads: int, D: int, dtype, device):
    return _torch().empty_strided((T, heads, D), (heads * D, D, 1), dtype=dtype, device=device)


def _qk_args(q_gain, k_gain, table, positions, T: int, D: int, interleaved: bool, norm: bool, device):
    """The arguments that norm and rotation share: gains and their type; table .. flags."""
    gdt, pq, pk = OQ_DTYPE_F32, None, None
    if q_gain is not None:
        gdt, pq = _mx_dtype(q_gain), _mx_rows(q_gain, (D,), q_gain.dtype, device, "q_gain")
        if k_gain is not None and k_gain.dtype is not q_gain.dtype:
            raise ValueError("q_gain and k_gain must have one type")
    if k_gain is not None:
        gdt, pk = _mx_dtype(k_gain), _mx_rows(k_gain, (D,), k_gain.dtype, device, "k_gain")
    pt, rows, rot, pp = None, 0, 0, None
    if table is not None:
        rows, half, two = table.shape if table.dim() == 3 else (0, 0, 0)
        if two != 2 or table.dtype is not _torch().float32 or table.device != device or not table.is_contiguous():
            raise ValueError(f"table must be contiguous float32 [positions, rot / 2, 2] on {device}")
        pt, rot = table.data_ptr(), 2 * half
        if positions is not None:
            pp = _ints(positions, (T,), device, "positions")
    elif positions is not None:
        raise ValueError("positions without a table")
    return pq, pk, gdt, pt, rows, rot, pp, (OQ_QK_INTERLEAVED if interleaved else 0) | (0 if norm else OQ_QK_NO_NORM)


def oq_qk_norm_rope(q, k=None, q_gain=None, k_gain=None, eps: float = 1e-6, table=None, positions=None,
                    interleaved: bool = False, norm: bool = True, q_out=None, k_out=None):
    """Norm for each head and rotation by position of q [T, heads, D] and k
    [T, kv_heads, D] (bf16/fp32, CUDA; a token's heads contiguous, tokens at any
    stride) -> (q_out, k_out) of the same types.  table: fp32 [positions, rot / 2,
    2] (cos, sin); positions: int32 [T], its row for each token (default: t).
    An output may be its input."""
    if q.dim() != 3 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [T, heads, D]")
    T, H, D = q.shape
    device, dtype, dt = q.device, q.dtype, _mx_dtype(q)
    pq, sq = _heads(q, None, D, device, "q")
    if q_out is None:
        q_out = _new_heads(T, H, D, dtype, device)
        pqo, sqo = q_out.data_ptr(), H * D
    else:
        if q_out.dtype is not dtype or q_out.shape != q.shape:
            raise ValueError("q_out must have q's type and shape")
        pqo, sqo = _heads(q_out, H, D, device, "q_out")
    pk = pko = None
    sk = sko = KH = 0
    if k is not None:
        if k.dtype is not dtype or k.dim() != 3 or k.shape[0] != T:
            raise ValueError("k must have q's type and tokens")
        KH = k.shape[1]
        pk, sk = _heads(k, None, D, device, "k")
        if k_out is None:
            k_out = _new_heads(T, KH, D, dtype, device)
            pko, sko = k_out.data_ptr(), KH * D
        else:
            if k_out.dtype is not dtype or k_out.shape != k.shape:
                raise ValueError("k_out must have k's type and shape")
            pko, sko = _heads(k_out, KH, D, device, "k_out")
    elif k_out is not None or k_gain is not None:
        raise ValueError("k_out or k_gain without k")
    g0, g1, gdt, pt, rows, rot, pp, flags = _qk_args(q_gain, k_gain, table, positions, T, D, interleaved, norm, device)
    _launch("oq_qk_norm_rope", device, pq, sq, H, pk, sk, KH, dt, T, D, g0, g1, gdt, eps, pt, rows, rot, pp, flags, pqo, sqo,
            pko, sko)
    return q_out, k_out


class Kv4:
    """Owns an oq_kv4* (a shape of attention over a 4-bit cache and its error word)."""

    def __init__(self, handle: int, lib, heads: int, kv_heads: int, head_dim: int, device: int):
        self._h = ctypes.c_void_p(handle)
        self._lib = lib
        self.device = device   # its index
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.groups = (kv_heads * head_dim + 127) // 128
        self.scale = head_dim ** -0.5
        self.workspaces = {}   # bytes of attention's workspace by (device, T, B, max_q, max_len)

    @property
    def handle(self):
        return self._h

    def cache(self, pages: int, device=None):
        """A new cache of so many pages of 128 tokens, zeroed: uint8 [pages, groups, 272, 64]."""
        torch = _torch()
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        return torch.zeros((pages, self.groups, 272, 64), dtype=torch.uint8, device=device)

    def close(self):
        if self._h:
            self._lib.oq_kv4_destroy(self._h)
            self._h = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def oq_kv4_create(heads: int, kv_heads: int, head_dim: int) -> Kv4:
    L = load_library()
    h = ctypes.c_void_p()
    _check(L.oq_kv4_create(heads, kv_heads, head_dim, ctypes.byref(h)), "oq_kv4_create")
    return Kv4(h.value, L, heads, kv_heads, head_dim, _torch().cuda.current_device())


def oq_kv4_destroy(kv: Kv4) -> None:
    kv.close()


def oq_kv4_cache_size(kv: Kv4, pages: int) -> int:
    return int(load_library().oq_kv4_cache_size(kv.handle, pages))


def _kv4_view(kv: Kv4, cache, page_table, cu, lens, device):
    """cache, pages, page table, its width, cu, lens, B as the C calls take them."""
    shape, table = cache.shape, page_table.shape
    if len(shape) != 4:
        raise ValueError("cache must be [pages, groups, 272, 64]")
    if len(table) != 2:
        raise ValueError("page_table must be [B, pages of a sequence]")
    B, width = table
    return (_mx_ptr(cache, (shape[0], kv.groups, 272, 64), device, "cache"), shape[0],
            _ints(page_table, table, device, "page_table"), width, _ints(cu, (B + 1,), device, "cu"),
            _ints(lens, (B,), device, "lens"), B)


def oq_kv4_append(kv: Kv4, q, k, v, cache, page_table, cu, lens, q_gain=None, k_gain=None, eps: float = 1e-6, table=None,
                  positions=None, interleaved: bool = False, norm: bool = True, q_out=None):
    """Keys and values [T, kv_heads, D] of new tokens to the cache, with the norm
    and rotation of oq_qk_norm_rope on queries and keys; q [T, heads, D] (or None)
    -> q_out bf16 [T, heads, D].  positions: default, each token's place in its
    sequence.  Rows of q_out that belong to no sequence are left alone (unset in a
    new tensor).  See include/orbitquant.h for cache, page_table, cu and lens."""
    torch = _torch()
    if k.dim() != 3 or not k.is_cuda:
        raise ValueError("k must be a CUDA tensor [T, kv_heads, D]")
    T, D, device, dt = k.shape[0], kv.head_dim, k.device, _mx_dtype(k)
    pk, sk = _heads(k, kv.kv_heads, D, device, "k")
    pv, sv = _heads(v, kv.kv_heads, D, device, "v")
    if v.dtype is not k.dtype or v.shape[0] != T:
        raise ValueError("v must have k's type and tokens")
    pq = pqo = None
    sq = 0
    if q is not None:
        if q.dtype is not k.dtype or q.dim() != 3 or q.shape[0] != T:
            raise ValueError("q must have k's type and tokens")
        pq, sq = _heads(q, kv.heads, D, device, "q")
        if q_out is None:
            q_out = _new_heads(T, kv.heads, D, torch.bfloat16, device)
            pqo = q_out.data_ptr()
        else:
            pqo = _mx_rows(q_out, (T, kv.heads, D), torch.bfloat16, device, "q_out")
    elif q_out is not None or q_gain is not None:
        raise ValueError("q_out or q_gain without q")
    g0, g1, gdt, pt, rows, rot, pp, flags = _qk_args(q_gain, k_gain, table, positions, T, D, interleaved, norm, device)
    _launch("oq_kv4_append", device, kv.handle, pq, sq, pk, sk, pv, sv, dt, T, g0, g1, gdt, eps, pt, rows, rot, pp, flags, pqo,
            *_kv4_view(kv, cache, page_table, cu, lens, device))
    return q_out


def oq_kv4_read(kv: Kv4, cache, page_table, cu, lens, T: int, dtype=None, k=None, v=None):
    """The values (fp32 by default, or bf16) that a call's T tokens have in the
    cache -> (k, v) [T, kv_heads, D]; NaN where a page is not there.  Rows of tokens
    without a place in the cache are left alone (unset in new tensors)."""
    torch = _torch()
    device, shape = cache.device, (T, kv.kv_heads, kv.head_dim)
    if device.type != "cuda":
        raise ValueError("cache must be a CUDA tensor")
    dtype = dtype if dtype is not None else k.dtype if k is not None else torch.float32
    if k is None:
        k = _new_heads(*shape, dtype, device)
    if v is None:
        v = _new_heads(*shape, dtype, device)
    _launch("oq_kv4_read", device, kv.handle, *_kv4_view(kv, cache, page_table, cu, lens, device), T,
            _mx_rows(k, shape, dtype, device, "k"), _mx_rows(v, shape, dtype, device, "v"), _mx_dtype(k))
    return k, v


def oq_kv4_attention_workspace_size(kv: Kv4, T: int, B: int, max_q: int, max_len: int) -> int:
    return int(load_library().oq_kv4_attention_workspace_size(kv.handle, T, B, max_q, max_len))


def oq_kv4_attention(kv: Kv4, q, cache, page_table, cu, lens, max_q: int, max_len: int = 0, scale=None, causal: bool = True,
                     window: int = 0, y=None, workspace=None):
    """softmax(scale q K^T + mask) V over the 4-bit cache: q [T, heads, D] bf16
    (CUDA, any token stride) -> y bf16 [T, heads, D].  max_q: the most tokens of a
    sequence in this call; max_len: about the longest sequence (default: what the
    page table holds); scale: default D^-0.5; window: 0, or how many tokens, itself
    among them, a token sees.  Rows of y that belong to no sequence, or to one's
    tokens past max_q, are left alone (unset in a new tensor)."""
    torch = _torch()
    if q.dim() != 3 or not q.is_cuda or q.dtype is not torch.bfloat16:
        raise ValueError("q must be a bfloat16 CUDA tensor [T, heads, D]")
    T, device, D = q.shape[0], q.device, kv.head_dim
    pq, sq = _heads(q, kv.heads, D, device, "q")
    view = _kv4_view(kv, cache, page_table, cu, lens, device)
    max_len = max_len or min(view[3] * OQ_KV4_PAGE, 0x7FFFFFFF)
    if y is None:
        y = _new_heads(T, kv.heads, D, torch.bfloat16, device)
        py = y.data_ptr()
    else:
        py = _mx_rows(y, (T, kv.heads, D), torch.bfloat16, device, "y")
    pw, nw = None, 0
    if workspace is None:
        sizes = (device.index, T, view[6], max_q, max_len)
        nw = kv.workspaces.get(sizes)
        if nw is None:
            with torch.cuda.device(device):   # (the split depends on the device's SMs)
                nw = oq_kv4_attention_workspace_size(kv, T, view[6], max_q, max_len)
            if len(kv.workspaces) >= 4096:
                kv.workspaces.clear()
            kv.workspaces[sizes] = nw
        if nw:
            workspace = torch.empty_strided((nw,), (1,), dtype=torch.uint8, device=device)
            pw = workspace.data_ptr()
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    else:
        pw, nw = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch("oq_kv4_attention", device, kv.handle, pq, sq, T, *view, max_q, max_len, kv.scale if scale is None else scale,
            OQ_ATTN_CAUSAL if causal else 0, window, py, pw, nw)
    return y


def oq_kv4_poll_error(kv: Kv4) -> None:
    with _torch().cuda.device(kv.device):
        _check(load_library().oq_kv4_poll_error(kv.handle), "oq_kv4_poll_error")


# ------------------------------------------------------------------ 4-bit weights with group scales
def oq_w4g_prepare(W, group: int, zeros: bool = False):
    """W [d_out, d_in] (fp32/bf16, CUDA) -> (codes [d_out, d_in rounded up to 128, / 2]
    uint8, scales [d_out, d_in / group] bf16, zeros uint8 or None)."""
    torch = _torch()
    if W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA matrix")
    d_out, d_in = W.shape
    if group not in (32, 64, 128) or d_in % group:
        raise ValueError("group must be 32, 64 or 128 and divide W's width")
    codes = torch.empty((d_out, (d_in + 127) // 128 * 64), dtype=torch.uint8, device=W.device)
    scales = torch.empty((d_out, d_in // group), dtype=torch.bfloat16, device=W.device)
    z = torch.empty((d_out, d_in // group), dtype=torch.uint8, device=W.device) if zeros else None
    _launch("oq_w4g_prepare", W.device, W.data_ptr(), _mx_dtype(W), d_out, d_in, group, codes.data_ptr(), scales.data_ptr(),
            None if z is None else z.data_ptr())
    return codes, scales, z


def oq_linear_w4g(x, codes, scales, zeros=None, group: int = 128, y=None, y_dtype=None):
    """x [T, d_in] (bf16/fp32, CUDA) times 4-bit weights with group scales (from
    oq_w4g_prepare) -> y [T, d_out] fp32 (or bf16)."""
    torch = _torch()
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA matrix")
    if codes.dim() != 2 or group not in (32, 64, 128) or x.shape[1] % group:
        raise ValueError("codes must be a matrix, group 32, 64 or 128 and divide x's width")
    T, d = x.shape
    n, device = codes.shape[0], x.device
    pc = _mx_ptr(codes, (n, (d + 127) // 128 * 64), device, "codes")
    ps = _mx_rows(scales, (n, d // group), torch.bfloat16, device, "scales")
    pz = None if zeros is None else _mx_ptr(zeros, (n, d // group), device, "zeros")
    if y is None:
        y = torch.empty_strided((T, n), (n, 1), dtype=torch.float32 if y_dtype is None else y_dtype, device=device)
        py = y.data_ptr()
    else:
        py = _mx_rows(y, (T, n), y.dtype if y_dtype is None else y_dtype, device, "y")
    _launch("oq_linear_w4g", device, x.data_ptr(), _mx_dtype(x), T, d, n, group, pc, ps, pz, py, _mx_dtype(y))
    return y


def oq_poll_error(layer: Layer) -> None:
    _check(load_library().oq_poll_error(layer.handle), "oq_poll_error")


def oq_check_wait_timeout(layer: Layer, limit_us: int) -> None:
    """Launch the bounded-wait self-test on the current stream (its wait runs
    out after limit_us microseconds; oq_poll_error then raises)."""
    torch = _torch()
    _check(load_library().oq_check_wait_timeout(
        layer.handle, int(limit_us), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)),
        "oq_check_wait_timeout")
