"""Python binding of libkq, the quantized weight-streaming GEMV library for
GB300 (sm_103a).

Argument marshalling only: every function here checks nothing the C library
does not check itself, turns torch tensors (device memory, owned by the
caller) and streams into pointers, calls the entry point of the same name in
libkq.so and raises KQError on a non-zero status.  All arithmetic runs in the
library's CUDA kernels (or, for the offline host quantizers, in its C++ host
code); there is no fallback of any kind.

If the shared library has not been built, importing this package fails with
an ImportError: build it with ``quantized_weight_streaming_gb300.build.build()``
(or ``__graft_entry__.build()``).
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libkq.so is not built ({LIB_PATH} missing); run quantized_weight_streaming_gb300.build.build()")

_lib = ctypes.CDLL(LIB_PATH)

KQ_OK = 0
KQ_ERR_INVALID_ARG = 1
KQ_ERR_SHAPE = 2
KQ_ERR_ALIGNMENT = 3
KQ_ERR_NONFINITE = 4
KQ_ERR_RANGE = 5
KQ_ERR_WORKSPACE = 6
KQ_ERR_CUDA = 7
KQ_ERR_TIMEOUT = 8
KQ_ERR_UNSUPPORTED = 9

KQ_Q8_0 = 0
KQ_PQ2_0 = 1
KQ_PTQ1_0 = 2  # storage format: kq_prepare transcodes it to PQ2_0 planes
KQ_SCALE4 = 3  # scale4_gs32
FORMATS = {"q8_0": KQ_Q8_0, "pq2_0": KQ_PQ2_0, "ptq1_0": KQ_PTQ1_0, "scale4": KQ_SCALE4}


class KQError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib.kq_last_error().decode()
        super().__init__(f"{where}: {_lib.kq_status_string(status).decode()} ({status}): {msg}")


class kq_qmat(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("had_block", ctypes.c_int32), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("signs", ctypes.c_void_p)]


KQ_SRC_PACKED = 0
KQ_SRC_INPUT_OF = 1
KQ_SRC_OUTPUT_OF = 2


class kq_link(ctypes.Structure):
    _fields_ = [("src", ctypes.c_int32), ("stage", ctypes.c_int32), ("of", ctypes.c_int64),
                ("alpha", ctypes.c_float), ("reserved", ctypes.c_int32)]


KQ_F32 = 0
KQ_F16 = 1
KQ_BF16 = 2


class kq_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class kq_kv_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class kq_qk_norm(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("d_rope", ctypes.c_void_p), ("rope_positions", ctypes.c_int64)]


class kq_rms(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("weight", ctypes.c_void_p)]


class kq_conv(ctypes.Structure):
    _fields_ = [("channels", ctypes.c_int32), ("width", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class kq_gdn_rule(ctypes.Structure):
    _fields_ = [("k_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("unit", ctypes.c_int32), ("gates", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("a_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_QP = ctypes.POINTER(kq_qmat)
_HP = ctypes.POINTER(kq_heads)
_CP = ctypes.POINTER(kq_kv_cache)
_NP = ctypes.POINTER(kq_qk_norm)
_RP = ctypes.POINTER(kq_rms)
_VP = ctypes.POINTER(kq_conv)
_GP = ctypes.POINTER(kq_gdn_rule)

# name -> (restype, argtypes); every symbol declared in include/kq.h
SIGNATURES = {
    "kq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kq_last_error": (ctypes.c_char_p, []),
    "kq_version": (ctypes.c_int, []),
    "kq_block_size": (_I64, [ctypes.c_int]),
    "kq_blocks_bytes": (_I64, [ctypes.c_int, _I64, _I64]),
    "kq_scale_stride": (_I64, [ctypes.c_int, _I64]),
    "kq_codes_bytes": (_I64, [ctypes.c_int, _I64, _I64]),
    "kq_scales_bytes": (_I64, [ctypes.c_int, _I64, _I64]),
    "kq_quantize_q8_0": (ctypes.c_int, [_P, _I64, _I64, _P]),
    "kq_quantize_pq2_0": (ctypes.c_int, [_P, _I64, _I64, _P]),
    "kq_quantize_ptq1_0": (ctypes.c_int, [_P, _I64, _I64, _P]),
    "kq_quantize_scale4": (ctypes.c_int, [_P, _I64, _I64, _P]),
    "kq_quantize_scale4_device": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "kq_gemv_scale4": (ctypes.c_int, [_QP, _P, _P, _P, _SZ, _P]),
    "kq_gemv_f16": (ctypes.c_int, [_QP, _P, _P, _P, _SZ, _P]),
    "kq_hadamard_blockwise_host": (ctypes.c_int, [_P, _P, _I64, _I64, _I32]),
    "kq_prepare": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _P, _P, _P]),
    "kq_quantize_q8_0_device": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "kq_quantize_pq2_0_device": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "kq_dequantize": (ctypes.c_int, [_QP, _P, _P]),
    "kq_embed": (ctypes.c_int, [_QP, _P, _I64, _P, _P]),
    "kq_hadamard_blockwise": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _P]),
    "kq_rotate_blockwise_host": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _P]),
    "kq_rotate_blockwise": (ctypes.c_int, [_P, _P, _I64, _I64, _I32, _P, _P]),
    "kq_gemv_workspace_bytes": (_SZ, [_QP, _I64]),
    "kq_gemv_q8_0": (ctypes.c_int, [_QP, _P, _P, _P, _SZ, _P]),
    "kq_gemv_pq2_0": (ctypes.c_int, [_QP, _P, _P, _P, _SZ, _P]),
    "kq_gemm_small_m": (ctypes.c_int, [_QP, _P, _I64, _P, _P, _SZ, _P]),
    "kq_gemm_tc": (ctypes.c_int, [_QP, _P, _I64, _P, _I32, _P, _SZ, _P]),
    "kq_gemm_tc_workspace_bytes": (_SZ, [_QP, _I64, _I32]),
    "kq_gemm_splitk": (ctypes.c_int, [_QP, _P, _I64, _P, _I32, _P, _SZ, _P]),
    "kq_gemm_splitk_workspace_bytes": (_SZ, [_QP, _I64, _I32]),
    "kq_gemm_splitk_noalloc": (ctypes.c_int, [_QP, _P, _I64, _P, _I32, _P]),
    "kq_gemm_splitk_noalloc_max_bytes": (_SZ, []),
    "kq_decode_plan_create": (ctypes.c_int, [_QP, _I64, ctypes.POINTER(_P)]),
    "kq_decode_plan_create_linked": (ctypes.c_int, [_QP, ctypes.POINTER(kq_link), _I64, ctypes.POINTER(_P)]),
    "kq_decode_plan_stages": (ctypes.c_int, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "kq_decode_plan_sizes": (ctypes.c_int, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "kq_decode_workspace_bytes": (_SZ, [_P]),
    "kq_decode_step": (ctypes.c_int, [_P, _P, _P, _P, _SZ, _P]),
    "kq_decode_step_host": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _SZ, _P]),
    "kq_decode_plan_destroy": (None, [_P]),
    "kq_stream_read": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P]),
    "kq_selftest_bounded_wait": (ctypes.c_int, [_I64, _P]),
    "kq_kv_block_bytes": (_I64, [_I32, _I32]),
    "kq_slot_map": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P]),
    "kq_rope_table_host": (ctypes.c_int, [_P, _I64, _I32, ctypes.c_double]),
    "kq_qk_norm_rope": (ctypes.c_int, [_NP, ctypes.c_int, _HP, _HP, _P, _I64, _HP, _HP, _P]),
    "kq_kv_append": (ctypes.c_int, [_NP, _CP, ctypes.c_int, _HP, _HP, _HP, _P, _P, _I64, _HP, _P]),
    "kq_kv_read": (ctypes.c_int, [_CP, _P, _I64, ctypes.c_int, _HP, _HP, _P]),
    "kq_attn_paged": (ctypes.c_int, [_CP, ctypes.c_int, _I32, _HP, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_float,
                                     _I64, _HP, _P, _SZ, _P]),
    "kq_attn_workspace_bytes": (_SZ, [_CP, _I32, _I64, _I64, _I64]),
    "kq_rms_norm": (ctypes.c_int, [_RP, ctypes.c_int, _HP, _HP, _HP, _I64, _HP, _QP, _P]),
    "kq_causal_conv": (ctypes.c_int, [_VP, ctypes.c_int, _HP, _P, _P, _P, _I64, _I64, _P, _I64, _HP, _P]),
    "kq_gdn": (ctypes.c_int, [_GP, ctypes.c_int, _HP, _HP, _HP, _P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I64, _P, _I64,
                              _HP, _P, _SZ, _P]),
    "kq_gdn_workspace_bytes": (_SZ, [_GP, ctypes.c_int, _I64, _I64, _I64]),
    "kq_sample": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P]),
    "kq_device_status": (ctypes.c_int, [ctypes.c_int]),
    "kq_set_pq2_0_consumer": (ctypes.c_int, [ctypes.c_int]),
    "kq_get_pq2_0_consumer": (ctypes.c_int, []),
    "kq_kernel_binary_version": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int)]),
}

for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib():
    return _lib


def _check(status, where):
    if status != KQ_OK:
        raise KQError(status, where)


def _ptr(t):
    """Address of a torch tensor, a numpy array or an integer (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


_raw_stream = None  # torch's lookup of the current stream's handle, once torch is imported


def _current_stream():
    """Handle of the current stream (torch.cuda.current_stream() builds a Stream object first: 3 us a call against 0.2)."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        torch.cuda.current_stream()  # initialises CUDA
        get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if get is None or device is None:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            _raw_stream = lambda: get(device())  # noqa: E731
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


# ---- layout ------------------------------------------------------------------

def kq_block_size(fmt):
    return _lib.kq_block_size(_fmt(fmt))


def kq_blocks_bytes(fmt, n, k):
    return _lib.kq_blocks_bytes(_fmt(fmt), n, k)


def kq_scale_stride(fmt, k):
    return _lib.kq_scale_stride(_fmt(fmt), k)


def kq_codes_bytes(fmt, n, k):
    return _lib.kq_codes_bytes(_fmt(fmt), n, k)


def kq_scales_bytes(fmt, n, k):
    return _lib.kq_scales_bytes(_fmt(fmt), n, k)


# ---- host quantizers (numpy in, numpy out) --------------------------------------

def kq_quantize_q8_0(w):
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    out = np.zeros(max(kq_blocks_bytes("q8_0", n, k), 1), dtype=np.uint8)
    _check(_lib.kq_quantize_q8_0(w.ctypes.data, n, k, out.ctypes.data), "kq_quantize_q8_0")
    return out[: n * (k // 32) * 34].reshape(n, k // 32, 34)


def kq_quantize_pq2_0(w_rot):
    w = np.ascontiguousarray(w_rot, dtype=np.float32)
    n, k = w.shape
    out = np.zeros(max(kq_blocks_bytes("pq2_0", n, k), 1), dtype=np.uint8)
    _check(_lib.kq_quantize_pq2_0(w.ctypes.data, n, k, out.ctypes.data), "kq_quantize_pq2_0")
    return out[: n * (k // 128) * 34].reshape(n, k // 128, 34)


def kq_quantize_scale4(w):
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    out = np.zeros(max(kq_blocks_bytes("scale4", n, k), 1), dtype=np.uint8)
    _check(_lib.kq_quantize_scale4(w.ctypes.data, n, k, out.ctypes.data), "kq_quantize_scale4")
    return out[: n * (k // 32) * 18].reshape(n, k // 32, 18)


def kq_quantize_ptq1_0(w_rot):
    w = np.ascontiguousarray(w_rot, dtype=np.float32)
    n, k = w.shape
    out = np.zeros(max(kq_blocks_bytes("ptq1_0", n, k), 1), dtype=np.uint8)
    _check(_lib.kq_quantize_ptq1_0(w.ctypes.data, n, k, out.ctypes.data), "kq_quantize_ptq1_0")
    return out[: n * (k // 128) * 28].reshape(n, k // 128, 28)


def kq_hadamard_blockwise_host(x, block=128):
    x = np.ascontiguousarray(x, dtype=np.float32)
    x2 = x.reshape(-1, x.shape[-1])
    out = np.empty_like(x2)
    _check(_lib.kq_hadamard_blockwise_host(x2.ctypes.data, out.ctypes.data, x2.shape[0], x2.shape[1], block),
           "kq_hadamard_blockwise_host")
    return out.reshape(x.shape)


# ---- device entry points (torch tensors) ------------------------------------------

class QMatrix:
    """A quantized matrix in device memory: torch tensors for the codes and
    scales planes plus the kq_qmat descriptor that points at them.  PQ2_0
    takes the rotation block (128, or the page's 1024) and an optional int8
    device tensor of k signs (kept referenced here)."""

    def __init__(self, fmt, n, k, device="cuda", had_block=None, signs=None):
        import torch

        self.fmt = _fmt(fmt)
        self.n, self.k = int(n), int(k)
        cb = kq_codes_bytes(self.fmt, n, k)
        sb = kq_scales_bytes(self.fmt, n, k)
        if cb <= 0 or sb <= 0:
            raise KQError(KQ_ERR_SHAPE, f"QMatrix({fmt}, {n}, {k})")
        self.codes = torch.empty(cb, dtype=torch.uint8, device=device)
        self.scales = torch.empty(sb // 2, dtype=torch.int16, device=device)
        if had_block is None:
            had_block = 128 if self.fmt == KQ_PQ2_0 else 0
        self.had_block = int(had_block)
        self.signs = signs
        self.desc = kq_qmat(self.fmt, self.had_block, self.n, self.k, self.codes.data_ptr(),
                            self.scales.data_ptr(), None if signs is None else signs.data_ptr())

    @property
    def nbytes(self):
        return self.codes.numel() + self.scales.numel() * 2

    @property
    def weight_bytes(self):
        """Bytes of the format itself (codes plus one fp16 scale per block)."""
        return self.codes.numel() + self.n * (self.k // kq_block_size(self.fmt)) * 2


def kq_prepare(W, d_blocks, stream=None, block_fmt=None):
    """Blocks (device memory) -> W's planes; block_fmt="ptq1_0" transcodes
    PTQ1_0 blocks into a PQ2_0 matrix."""
    fmt = W.fmt if block_fmt is None else _fmt(block_fmt)
    _check(_lib.kq_prepare(fmt, _ptr(d_blocks), W.n, W.k, W.codes.data_ptr(), W.scales.data_ptr(), _stream(stream)),
           "kq_prepare")


def kq_quantize_q8_0_device(W, d_w, stream=None):
    _check(_lib.kq_quantize_q8_0_device(_ptr(d_w), W.n, W.k, W.codes.data_ptr(), W.scales.data_ptr(),
                                        _stream(stream)), "kq_quantize_q8_0_device")


def kq_quantize_pq2_0_device(W, d_w_rot, stream=None):
    _check(_lib.kq_quantize_pq2_0_device(_ptr(d_w_rot), W.n, W.k, W.codes.data_ptr(), W.scales.data_ptr(),
                                         _stream(stream)), "kq_quantize_pq2_0_device")


def kq_quantize_scale4_device(W, d_w, stream=None):
    _check(_lib.kq_quantize_scale4_device(_ptr(d_w), W.n, W.k, W.codes.data_ptr(), W.scales.data_ptr(),
                                          _stream(stream)), "kq_quantize_scale4_device")


def kq_embed(E, d_ids, count, d_out, stream=None):
    """Rows d_ids of the quantized table E, dequantized (and inverse-rotated for PQ2_0)."""
    _check(_lib.kq_embed(ctypes.byref(E.desc), _ptr(d_ids), count, _ptr(d_out), _stream(stream)), "kq_embed")


def kq_dequantize(W, d_out, stream=None):
    _check(_lib.kq_dequantize(ctypes.byref(W.desc), _ptr(d_out), _stream(stream)), "kq_dequantize")


def kq_hadamard_blockwise(d_in, d_out, rows, k, block=128, stream=None):
    _check(_lib.kq_hadamard_blockwise(_ptr(d_in), _ptr(d_out), rows, k, block, _stream(stream)),
           "kq_hadamard_blockwise")


def kq_rotate_blockwise(d_in, d_out, rows, k, block, d_signs=None, stream=None):
    _check(_lib.kq_rotate_blockwise(_ptr(d_in), _ptr(d_out), rows, k, block, _ptr(d_signs), _stream(stream)),
           "kq_rotate_blockwise")


def kq_rotate_blockwise_host(x, block, signs=None):
    x = np.ascontiguousarray(x, dtype=np.float32)
    x2 = x.reshape(-1, x.shape[-1])
    out = np.empty_like(x2)
    sg = None if signs is None else np.ascontiguousarray(signs, dtype=np.int8)
    _check(_lib.kq_rotate_blockwise_host(x2.ctypes.data, out.ctypes.data, x2.shape[0], x2.shape[1], block,
                                         None if sg is None else sg.ctypes.data), "kq_rotate_blockwise_host")
    return out.reshape(x.shape)


def kq_gemv_workspace_bytes(W, m=1):
    return _lib.kq_gemv_workspace_bytes(ctypes.byref(W.desc), m)


def kq_gemm_splitk_workspace_bytes(W, m, splits):
    return _lib.kq_gemm_splitk_workspace_bytes(ctypes.byref(W.desc), m, splits)


def _ws(ws):
    if ws is None:
        return None, 0
    return _ptr(ws), ws.numel() * ws.element_size()


def kq_gemv_q8_0(W, d_x, d_y, ws=None, stream=None):
    p, nb = _ws(ws)
    _check(_lib.kq_gemv_q8_0(ctypes.byref(W.desc), _ptr(d_x), _ptr(d_y), p, nb, _stream(stream)), "kq_gemv_q8_0")


def kq_gemv_scale4(W, d_x, d_y, ws=None, stream=None):
    p, nb = _ws(ws)
    _check(_lib.kq_gemv_scale4(ctypes.byref(W.desc), _ptr(d_x), _ptr(d_y), p, nb, _stream(stream)), "kq_gemv_scale4")


def kq_gemv_f16(W, d_x16, d_y16, ws=None, stream=None):
    """The fp16 chain: fp16 activation in, fp16 output (any format)."""
    p, nb = _ws(ws)
    _check(_lib.kq_gemv_f16(ctypes.byref(W.desc), _ptr(d_x16), _ptr(d_y16), p, nb, _stream(stream)), "kq_gemv_f16")


def kq_gemv_pq2_0(W, d_x, d_y, ws=None, stream=None):
    p, nb = _ws(ws)
    _check(_lib.kq_gemv_pq2_0(ctypes.byref(W.desc), _ptr(d_x), _ptr(d_y), p, nb, _stream(stream)), "kq_gemv_pq2_0")


def kq_gemm_small_m(W, d_X, m, d_Y, ws=None, stream=None):
    p, nb = _ws(ws)
    _check(_lib.kq_gemm_small_m(ctypes.byref(W.desc), _ptr(d_X), m, _ptr(d_Y), p, nb, _stream(stream)),
           "kq_gemm_small_m")


def kq_gemm_tc_workspace_bytes(W, m, splits=0):
    return _lib.kq_gemm_tc_workspace_bytes(ctypes.byref(W.desc), m, splits)


def kq_gemm_tc(W, d_X, m, d_Y, splits=0, ws=None, stream=None):
    """Small-batch GEMM on the tensor cores (tcgen05)."""
    p, nb = _ws(ws)
    _check(_lib.kq_gemm_tc(ctypes.byref(W.desc), _ptr(d_X), m, _ptr(d_Y), splits, p, nb, _stream(stream)),
           "kq_gemm_tc")


def kq_gemm_splitk(W, d_X, m, d_Y, splits, ws=None, stream=None):
    p, nb = _ws(ws)
    _check(_lib.kq_gemm_splitk(ctypes.byref(W.desc), _ptr(d_X), m, _ptr(d_Y), splits, p, nb, _stream(stream)),
           "kq_gemm_splitk")


def kq_kernel_binary_version():
    v = ctypes.c_int()
    _check(_lib.kq_kernel_binary_version(ctypes.byref(v)), "kq_kernel_binary_version")
    return v.value


def kq_gemm_splitk_noalloc(W, d_X, m, d_Y, splits, stream=None):
    """Split-K GEMM whose partial sums use the library's static device scratch
    (no workspace argument, no allocation)."""
    _check(_lib.kq_gemm_splitk_noalloc(ctypes.byref(W.desc), _ptr(d_X), m, _ptr(d_Y), splits, _stream(stream)),
           "kq_gemm_splitk_noalloc")


def kq_gemm_splitk_noalloc_max_bytes():
    return _lib.kq_gemm_splitk_noalloc_max_bytes()


def kq_selftest_bounded_wait(limit_cycles, stream=None):
    _check(_lib.kq_selftest_bounded_wait(int(limit_cycles), _stream(stream)), "kq_selftest_bounded_wait")


def kq_stream_read(d_src, nbytes, d_sink, stage_bytes=34816, stages=4, stream=None):
    """Read-only streaming control: stream nbytes of d_src once through shared
    memory; XORs the XOR of its 32-bit words into d_sink[0]."""
    _check(_lib.kq_stream_read(_ptr(d_src), nbytes, stage_bytes, stages, _ptr(d_sink), _stream(stream)),
           "kq_stream_read")


def kq_device_status(clear=True):
    return _lib.kq_device_status(1 if clear else 0)


# ---- attention between the projections -----------------------------------------------

def kq_kv_block_bytes(page_size, head_dim):
    return _lib.kq_kv_block_bytes(page_size, head_dim)


class KVCache:
    """A paged 4-bit key/value cache of one layer: a torch tensor of
    [pages, kv_heads, kq_kv_block_bytes] bytes (`data`, or a new zeroed one)
    and the descriptor that points at it."""

    def __init__(self, pages, page_size, kv_heads, head_dim, data=None, device="cuda"):
        import torch

        nb = kq_kv_block_bytes(page_size, head_dim)
        if nb <= 0 or pages < 1 or kv_heads < 1:
            raise KQError(KQ_ERR_SHAPE, f"KVCache({pages}, {page_size}, {kv_heads}, {head_dim})")
        if data is None:
            data = torch.zeros(pages, kv_heads, nb, dtype=torch.uint8, device=device)
        elif data.numel() * data.element_size() != pages * kv_heads * nb or not data.is_contiguous():
            raise KQError(KQ_ERR_SHAPE, f"KVCache data: {pages} x {kv_heads} x {nb} contiguous bytes are needed")
        self.data = data
        self.pages, self.page_size, self.kv_heads, self.head_dim = int(pages), int(page_size), int(kv_heads), int(head_dim)
        self.desc = kq_kv_cache(data.data_ptr(), self.pages, self.page_size, self.kv_heads, self.head_dim, 0)
        self._ref = ctypes.byref(self.desc)


def _floats(t, name, shape):
    """Address of a contiguous fp32 tensor that fills `shape` in its last dimensions (None -> NULL)."""
    if t is None:
        return None
    if str(t.dtype) == "torch.float32" and t.is_contiguous() and t.dim() >= len(shape) and \
            tuple(t.shape[t.dim() - len(shape):]) == shape:
        return t.data_ptr()
    raise KQError(KQ_ERR_SHAPE, f"{name}: a contiguous fp32 tensor of {shape} is needed, not {tuple(t.shape)} {t.dtype}")


class QKNorm:
    """A kq_qk_norm descriptor and the device tensors it points at: fp32
    weights [head_dim] (None: ones), the fp32 rotation table [positions,
    rope_dim] (kq_rope_table_host).  norm=False leaves the norm out."""

    def __init__(self, q_heads, kv_heads, head_dim, rope_dim=0, q_weight=None, k_weight=None, rope=None, eps=1e-6,
                 interleaved=False, norm=True):
        self.q_weight, self.k_weight, self.rope = q_weight, k_weight, rope
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        rows = 0 if rope is None else rope.shape[0]
        self.desc = kq_qk_norm(q_heads, kv_heads, head_dim, rope_dim, int(interleaved), int(norm), eps, 0,
                               _floats(q_weight, "q_weight", (head_dim,)), _floats(k_weight, "k_weight", (head_dim,)),
                               _floats(rope, "rope", (rows, rope_dim)) if rope_dim else None, rows)
        self._ref = ctypes.byref(self.desc)


_DTYPES = {}  # torch dtype -> (kq_dtype or -1, whether it is int32), filled on first use


def _kind(dtype):
    k = _DTYPES.get(dtype)
    if k is None:
        names = {"torch.float32": KQ_F32, "torch.float16": KQ_F16, "torch.bfloat16": KQ_BF16}
        k = _DTYPES[dtype] = (names.get(str(dtype), -1), str(dtype) == "torch.int32")
    return k


def _dtype(t):
    return _kind(t.dtype)[0]


def _heads(t, heads, head_dim, name, like=None):
    """kq_heads of a [tokens, heads, head_dim] view whose innermost dimension is contiguous (None -> NULL)."""
    if t is None:
        return None
    shape = t.shape
    if len(shape) == 3:
        n, h, d = shape
        st, sh, sd = t.stride()
        if h == heads and d == head_dim and (sd == 1 or n == 0) and \
                (like is None or (n == like.shape[0] and t.dtype is like.dtype)):
            return kq_heads(t.data_ptr(), st if n > 1 else 0, sh if h > 1 else 0)
    raise KQError(KQ_ERR_SHAPE, f"{name} {tuple(shape)} {t.dtype} strides {t.stride()}: [tokens, {heads}, {head_dim}] "
                                "of one type for all, innermost contiguous, is needed")


def _ints(t, count, name):
    """Address of a contiguous int32 tensor of at least `count` elements."""
    if t is None:
        return None
    if _kind(t.dtype)[1] and t.is_contiguous() and t.numel() >= count:
        return t.data_ptr()
    raise KQError(KQ_ERR_SHAPE, f"{name}: a contiguous int32 tensor of {count} elements is needed, not "
                                f"{tuple(t.shape)} {t.dtype}")


def kq_slot_map(d_cached, d_new, page_size, d_free_pages, d_block_table, d_q_start, d_kv_len, d_positions, d_slots,
                d_pages_used, stream=None):
    """Block tables and slot maps of a step; d_block_table [requests, table_stride], the capacity of the token arrays is
    d_slots' length."""
    r, t = d_cached.numel(), d_slots.numel()
    if d_block_table.dim() != 2 or d_block_table.shape[0] < r:
        raise KQError(KQ_ERR_SHAPE, f"block table {tuple(d_block_table.shape)} for {r} requests")
    _check(_lib.kq_slot_map(_ints(d_cached, r, "d_cached"), _ints(d_new, r, "d_new"), r, page_size,
                            _ints(d_free_pages, 0, "d_free_pages"), 0 if d_free_pages is None else d_free_pages.numel(),
                            _ints(d_block_table, 0, "d_block_table"), d_block_table.shape[1],
                            _ints(d_q_start, r + 1, "d_q_start"), _ints(d_kv_len, r, "d_kv_len"),
                            _ints(d_positions, t, "d_positions"), _ints(d_slots, t, "d_slots"), t,
                            _ints(d_pages_used, 1, "d_pages_used"), _stream(stream)), "kq_slot_map")


def kq_rope_table_host(positions, rope_dim, base):
    out = np.empty((positions, rope_dim), dtype=np.float32)
    _check(_lib.kq_rope_table_host(out.ctypes.data, positions, rope_dim, base), "kq_rope_table_host")
    return out


def kq_qk_norm_rope(p, q, k, d_positions, q_out, k_out, stream=None):
    """Norm and rotation of q [tokens, q_heads, D] and k [tokens, kv_heads, D] (strided views) into q_out, k_out."""
    hq, hk, d, t = p.q_heads, p.kv_heads, p.head_dim, q.shape[0]
    _check(_lib.kq_qk_norm_rope(p._ref, _dtype(q), _heads(q, hq, d, "q"), _heads(k, hk, d, "k", q),
                                _ints(d_positions, t, "d_positions"), t, _heads(q_out, hq, d, "q_out", q),
                                _heads(k_out, hk, d, "k_out", q), _stream(stream)), "kq_qk_norm_rope")


def kq_kv_append(p, cache, q, k, v, d_positions, d_slots, q_out, stream=None):
    """Norm and rotation of q into q_out; keys (normed, rotated) and values into the cache at d_slots, in 4 bits.
    q and q_out may be None."""
    hq, hk, d, t = p.q_heads, p.kv_heads, p.head_dim, k.shape[0]
    _check(_lib.kq_kv_append(p._ref, cache._ref, _dtype(k), _heads(q, hq, d, "q", k), _heads(k, hk, d, "k"),
                             _heads(v, hk, d, "v", k), _ints(d_positions, t, "d_positions"), _ints(d_slots, t, "d_slots"), t,
                             _heads(q_out, hq, d, "q_out", k), _stream(stream)), "kq_kv_append")


def kq_kv_read(cache, d_slots, k_out, v_out, stream=None):
    """What the cache holds at d_slots, as values: k_out, v_out [count, kv_heads, D]."""
    h, d, n = cache.kv_heads, cache.head_dim, k_out.shape[0]
    _check(_lib.kq_kv_read(cache._ref, _ints(d_slots, n, "d_slots"), n, _dtype(k_out), _heads(k_out, h, d, "k_out"),
                           _heads(v_out, h, d, "v_out", k_out), _stream(stream)), "kq_kv_read")


def kq_attn_workspace_bytes(cache, q_heads, requests, tokens, max_new):
    return _lib.kq_attn_workspace_bytes(cache._ref, q_heads, requests, tokens, max_new)


def kq_attn_paged(cache, q, d_q_start, d_kv_len, d_block_table, out, scale, max_new, window=0, ws=None, stream=None):
    """Attention of the step's new tokens q [tokens, q_heads, D] over the cache, causal, optionally over a sliding
    window; at most max_new new tokens a request."""
    p, nb = _ws(ws)
    r, shape, table, d = d_kv_len.numel(), q.shape, d_block_table.shape, cache.head_dim
    if len(table) != 2 or table[0] < r or len(shape) != 3:
        raise KQError(KQ_ERR_SHAPE, f"block table {tuple(table)} for {r} requests, q {tuple(shape)}")
    hq = shape[1]
    _check(_lib.kq_attn_paged(cache._ref, _dtype(q), hq, _heads(q, hq, d, "q"), _ints(d_q_start, r + 1, "d_q_start"),
                              _ints(d_kv_len, r, "d_kv_len"), _ints(d_block_table, 0, "d_block_table"), table[1], r,
                              shape[0], max_new, scale, window, _heads(out, hq, d, "out", q), p, nb, _stream(stream)),
           "kq_attn_paged")


# ---- norms, gated-delta layers and sampling ------------------------------------------

class RMSNorm:
    """A kq_rms descriptor and the fp32 weight [dim] (None: ones) that it points at."""

    def __init__(self, heads, dim, weight=None, eps=1e-6):
        self.weight, self.heads, self.dim = weight, heads, dim
        self.desc = kq_rms(heads, dim, eps, 0, _floats(weight, "weight", (dim,)))
        self._ref = ctypes.byref(self.desc)


def kq_rms_norm(p, x, out=None, residual=None, gate=None, out_q8=None, stream=None):
    """RMS norm of the rows of x [tokens, heads, dim] (strided views): of x + residual, which residual then holds, where one
    is given; times silu(gate) where one is.  To out, to the Q8_0 planes of out_q8 (a QMatrix of tokens * heads rows), or
    both."""
    h, d, t = p.heads, p.dim, x.shape[0]
    _check(_lib.kq_rms_norm(p._ref, _dtype(x), _heads(x, h, d, "x"), _heads(residual, h, d, "residual", x),
                            _heads(gate, h, d, "gate", x), t, _heads(out, h, d, "out", x),
                            None if out_q8 is None else ctypes.byref(out_q8.desc), _stream(stream)), "kq_rms_norm")


class CausalConv:
    """A kq_conv descriptor and the fp32 tensors that it points at: weight [channels, width], bias [channels] or None."""

    def __init__(self, weight, bias=None, silu=True):
        if weight.dim() != 2:
            raise KQError(KQ_ERR_SHAPE, f"weight {tuple(weight.shape)}: [channels, width] is needed")
        self.weight, self.bias = weight, bias
        self.channels, self.width = weight.shape
        self.desc = kq_conv(self.channels, self.width, int(silu), 0, _floats(weight, "weight", tuple(weight.shape)),
                            _floats(bias, "bias", (self.channels,)))
        self._ref = ctypes.byref(self.desc)


def _wide_rows(t, wide, name, like=None):
    """kq_heads of a [tokens, wide] view whose rows are contiguous."""
    shape = t.shape
    if len(shape) == 2:
        n, c = shape
        st, sc = t.stride()
        if c == wide and (sc == 1 or n == 0) and (like is None or (n == like.shape[0] and t.dtype is like.dtype)):
            return kq_heads(t.data_ptr(), st if n > 1 else 0, 0)
    raise KQError(KQ_ERR_SHAPE, f"{name} {tuple(shape)} {t.dtype} strides {t.stride()}: [tokens, {wide}] of one type for "
                                "all, innermost contiguous, is needed")


def _states(t, like, shape, name):
    """(address, slots) of a contiguous tensor [slots, *shape] of the type `like`."""
    if t.dtype is like and t.is_contiguous() and tuple(t.shape[1:]) == shape:
        return t.data_ptr(), t.shape[0]
    raise KQError(KQ_ERR_SHAPE, f"{name} {tuple(t.shape)} {t.dtype}: a contiguous {like} tensor [slots, "
                                f"{', '.join(map(str, shape))}] is needed")


def kq_causal_conv(p, x, d_q_start, d_kv_len, d_slot, state, out, stream=None):
    """The short causal convolution of x [tokens, channels] into out, request by request; state [slots, width - 1,
    channels] of x's type holds each slot's last inputs.  d_kv_len may be None: then every state goes on."""
    r, t, c = d_slot.numel(), x.shape[0], p.channels
    at, slots = _states(state, x.dtype, (p.width - 1, c), "state")
    _check(_lib.kq_causal_conv(p._ref, _dtype(x), _wide_rows(x, c, "x"), _ints(d_q_start, r + 1, "d_q_start"),
                               _ints(d_kv_len, r, "d_kv_len"), _ints(d_slot, r, "d_slot"), r, t, at, slots,
                               _wide_rows(out, c, "out", x), _stream(stream)), "kq_causal_conv")


class GatedDelta:
    """A kq_gdn_rule descriptor and the fp32 tensors a_log, dt_bias [v_heads] that it points at (both None: the gates given
    to kq_gdn are log decays and strengths as they are).  scale: None for head_dim ** -0.5."""

    def __init__(self, k_heads, v_heads, head_dim, a_log=None, dt_bias=None, unit=True, eps=1e-6, scale=None):
        self.a_log, self.dt_bias = a_log, dt_bias
        self.k_heads, self.v_heads, self.head_dim = k_heads, v_heads, head_dim
        self.desc = kq_gdn_rule(k_heads, v_heads, head_dim, int(unit), int(a_log is not None), eps,
                                head_dim ** -0.5 if scale is None else scale, 0, _floats(a_log, "a_log", (v_heads,)),
                                _floats(dt_bias, "dt_bias", (v_heads,)))
        self._ref = ctypes.byref(self.desc)


def kq_gdn_workspace_bytes(p, dtype, requests, tokens, max_new):
    """Workspace bytes of kq_gdn; dtype a torch dtype."""
    return _lib.kq_gdn_workspace_bytes(p._ref, _kind(dtype)[0], requests, tokens, max_new)


def _gate(t, heads, name, like):
    """(address, token stride) of a [tokens, heads] view whose rows are contiguous."""
    if t.dim() == 2 and t.shape[0] == like.shape[0] and t.shape[1] == heads and t.dtype is like.dtype and \
            (t.stride(1) == 1 or heads == 1 or t.shape[0] == 0):
        return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0
    raise KQError(KQ_ERR_SHAPE, f"{name} {tuple(t.shape)} {t.dtype} strides {t.stride()}: [{like.shape[0]}, {heads}] of "
                                "q's type, innermost contiguous, is needed")


_FLOAT32 = None


def kq_gdn(p, q, k, v, a, b, d_q_start, d_kv_len, d_slot, state, out, max_new, ws=None, stream=None):
    """The gated delta rule over the step's new tokens: q, k [tokens, k_heads, D], v, out [tokens, v_heads, D], gates a, b
    [tokens, v_heads]; state fp32 [slots, v_heads, D, D], updated.  d_kv_len may be None: then every state goes on."""
    global _FLOAT32
    if _FLOAT32 is None:
        import torch

        _FLOAT32 = torch.float32
    hk, hv, d, r, t = p.k_heads, p.v_heads, p.head_dim, d_slot.numel(), q.shape[0]
    at, slots = _states(state, _FLOAT32, (hv, d, d), "state")
    a_at, a_stride = _gate(a, hv, "a", q)
    b_at, b_stride = _gate(b, hv, "b", q)
    w, nb = _ws(ws)
    _check(_lib.kq_gdn(p._ref, _dtype(q), _heads(q, hk, d, "q"), _heads(k, hk, d, "k", q), _heads(v, hv, d, "v", q), a_at,
                       a_stride, b_at, b_stride, _ints(d_q_start, r + 1, "d_q_start"), _ints(d_kv_len, r, "d_kv_len"),
                       _ints(d_slot, r, "d_slot"), r, t, max_new, at, slots, _heads(out, hv, d, "out", q), w, nb,
                       _stream(stream)), "kq_gdn")


def _per_row(t, rows, name):
    if t is None:
        return None
    if _kind(t.dtype)[0] == KQ_F32 and t.is_contiguous() and t.numel() >= rows:
        return t.data_ptr()
    raise KQError(KQ_ERR_SHAPE, f"{name}: a contiguous fp32 tensor of {rows} elements is needed, not {tuple(t.shape)} {t.dtype}")


def kq_sample(logits, u, d_token, d_prob=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """A token from each row of logits [rows, vocab] (rows may be strided) by the random numbers u [rows]; the settings are
    device tensors [rows] (top_k int32, the others fp32) or None."""
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise KQError(KQ_ERR_SHAPE, f"logits {tuple(logits.shape)} strides {logits.stride()}: [rows, vocab], innermost "
                                    "contiguous, is needed")
    r, v = logits.shape
    _check(_lib.kq_sample(_dtype(logits), logits.data_ptr(), logits.stride(0) if r > 1 else 0, r, v,
                          _per_row(temperature, r, "temperature"), _ints(top_k, r, "top_k"), _per_row(top_p, r, "top_p"),
                          _per_row(min_p, r, "min_p"), _per_row(u, r, "u"), _ints(d_token, r, "d_token"),
                          _per_row(d_prob, r, "d_prob"), _stream(stream)), "kq_sample")


KQ_PQ2_0_MMA_SYNC = 0
KQ_PQ2_0_TCGEN05 = 1


def kq_set_pq2_0_consumer(consumer):
    """Selects the consumer of PQ2_0 products at one activation row
    (KQ_PQ2_0_MMA_SYNC, the default, or KQ_PQ2_0_TCGEN05); process-wide."""
    _check(_lib.kq_set_pq2_0_consumer(int(consumer)), "kq_set_pq2_0_consumer")


def kq_get_pq2_0_consumer():
    return _lib.kq_get_pq2_0_consumer()


class DecodePlan:
    """kq_decode_plan_create (or, with links, kq_decode_plan_create_linked) /
    kq_decode_step / kq_decode_plan_destroy.  links: one (src, stage, of,
    alpha) tuple per matrix."""

    def __init__(self, mats, links=None):
        self.mats = list(mats)
        arr = (kq_qmat * len(self.mats))(*[m.desc for m in self.mats])
        h = ctypes.c_void_p()
        if links is None:
            _check(_lib.kq_decode_plan_create(arr, len(self.mats), ctypes.byref(h)), "kq_decode_plan_create")
        else:
            links = list(links)
            la = (kq_link * len(links))(*[kq_link(int(src), int(stage), int(of), float(alpha), 0)
                                          for src, stage, of, alpha in links])
            _check(_lib.kq_decode_plan_create_linked(arr, la, len(links), ctypes.byref(h)),
                   "kq_decode_plan_create_linked")
        self.handle = h
        st, ns = _I32(), _I32()
        _check(_lib.kq_decode_plan_stages(h, ctypes.byref(st), ctypes.byref(ns)), "kq_decode_plan_stages")
        self.stages, self.split_matrices = st.value, ns.value
        xf, yf, wb = _I64(), _I64(), _I64()
        _check(_lib.kq_decode_plan_sizes(h, ctypes.byref(xf), ctypes.byref(yf), ctypes.byref(wb)),
               "kq_decode_plan_sizes")
        self.x_floats, self.y_floats, self.weight_bytes = xf.value, yf.value, wb.value
        self.workspace_bytes = _lib.kq_decode_workspace_bytes(h)

    def step(self, d_x_packed, d_y_packed, ws=None, stream=None):
        p, nb = _ws(ws)
        _check(_lib.kq_decode_step(self.handle, _ptr(d_x_packed), _ptr(d_y_packed), p, nb, _stream(stream)),
               "kq_decode_step")

    def step_host(self, h_x_packed, h_y_packed, d_x_packed, d_y_packed, ws=None, stream=None):
        """kq_decode_step_host: host (ideally pinned) CPU tensors in and out,
        through the given device buffers; asynchronous on `stream`.  A pinned
        h_x_packed is read by the kernel in place (d_x_packed is then left
        unwritten), and a one-stage plan writes a pinned h_y_packed directly
        (d_y_packed is then left unwritten)."""
        p, nb = _ws(ws)
        _check(_lib.kq_decode_step_host(self.handle, _ptr(h_x_packed), _ptr(h_y_packed), _ptr(d_x_packed),
                                        _ptr(d_y_packed), p, nb, _stream(stream)), "kq_decode_step_host")

    def close(self):
        if self.handle:
            _lib.kq_decode_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
