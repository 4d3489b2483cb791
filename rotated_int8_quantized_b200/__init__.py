"""INT8 ConvRot linear layer on NVIDIA B200 (sm_100a).

Thin ctypes binding over ``libconvrot.so`` (C ABI in ``include/convrot.h``).
Every function here only marshals torch tensors into device pointers and
sizes and calls the C entry point of the same name; all arithmetic runs in
the library's CUDA kernels.  There is no CPU fallback: if the library is
missing or the device is not a B200, calls raise.

Typical use::

    w = quantize_weight(w_bf16)                 # offline, QuantizedWeight
    ws = make_workspace(m, w)                   # zero-filled scratch
    y = linear_int8(x_bf16, w, ws)              # BF16 [m, n]
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libconvrot.so")
GROUP = 256

_STATUS = {
    0: "CONVROT_OK", 1: "CONVROT_ERR_INVALID_ARG", 2: "CONVROT_ERR_ALIGNMENT",
    3: "CONVROT_ERR_UNSUPPORTED_SHAPE", 4: "CONVROT_ERR_UNSUPPORTED_ARCH",
    5: "CONVROT_ERR_WORKSPACE", 6: "CONVROT_ERR_CUDA", 7: "CONVROT_ERR_DEVICE_TIMEOUT",
    8: "CONVROT_WARN_INEXACT_DOMAIN",
}


class ConvrotError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s" % (where, _STATUS.get(status, "status %d" % status)))


class convrot_weight_t(ctypes.Structure):
    """Mirror of the C struct: a view of (q int8 [n,k], scale fp32 [n])."""
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int32)]


class convrot_linear_job_t(ctypes.Structure):
    """Mirror of the C struct: one linear of a batched call."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("w", ctypes.POINTER(convrot_weight_t)),
                ("y_bf16", ctypes.c_void_p), ("bias_bf16", ctypes.c_void_p)]


class convrot_weight4_t(ctypes.Structure):
    """Mirror of the C struct: packed INT4 weight (q uint8 [n, k/2], scale fp32 [n])."""
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int32)]


class convrot_linear4_job_t(ctypes.Structure):
    """Mirror of the C struct: one W4A8 linear of a call."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("w", ctypes.POINTER(convrot_weight4_t)),
                ("y_bf16", ctypes.c_void_p), ("bias_bf16", ctypes.c_void_p)]


class convrot_conv2d_t(ctypes.Structure):
    """Mirror of the C struct: convolution geometry (NHWC input)."""
    _fields_ = [(f, ctypes.c_int32) for f in ("n", "h", "w", "c", "kh", "kw", "stride", "pad", "dilation")]


class convrot_conv2d_plan_t(ctypes.Structure):
    """Mirror of the C struct: how the im2col gather of a convolution runs."""
    _fields_ = [("tiled", ctypes.c_int32), ("th", ctypes.c_int32), ("tw", ctypes.c_int32), ("rh", ctypes.c_int32),
                ("rw", ctypes.c_int32), ("tiles", ctypes.c_int64), ("buf_bytes", ctypes.c_int64)]


class convrot_gemm_plan_t(ctypes.Structure):
    """Mirror of the C struct: how the GEMM kernel tiles a product."""
    _fields_ = [(f, ctypes.c_int32) for f in ("njobs", "swap", "bn", "grid", "full_waves", "full_tiles",
                                               "split_ways", "split_pieces", "rep", "stages", "tmem_cols",
                                               "slots")] + \
               [(f, ctypes.c_int64) for f in ("tail_units", "smem_bytes", "ws_bytes")] + \
               [(f, ctypes.c_int32 * 8) for f in ("tiles_a", "tiles_b", "group_a", "kbpt", "tile_base")] + \
               [("unit0", ctypes.c_int64 * 8)]


class convrot_gemm_job_t(ctypes.Structure):
    """Mirror of the C struct: one product of a batched GEMM call."""
    _fields_ = [("xq", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("w", ctypes.POINTER(convrot_weight_t)),
                ("y_bf16", ctypes.c_void_p), ("acc", ctypes.c_void_p), ("bias_bf16", ctypes.c_void_p)]


class convrot_kv8_t(ctypes.Structure):
    """Mirror of the C struct: a view of a paged INT8 key/value cache."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale")] + [("pages", ctypes.c_int64)] + \
               [(f, ctypes.c_int32) for f in ("kv_heads", "page_tokens", "head_dim")]


class convrot_rope_t(ctypes.Structure):
    """Mirror of the C struct: the position rotation."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("adjacent", ctypes.c_int32), ("axis", ctypes.c_void_p), ("axes", ctypes.c_int32)]


class convrot_kv8_seqs_t(ctypes.Structure):
    """Mirror of the C struct: the sequences of a step."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("page_table", "kv_len", "cu")] + [("tokens", ctypes.c_int64)] + \
               [(f, ctypes.c_int32) for f in ("batch", "max_pages")]


def _rows_fields(*names):
    return [f for n in names for f in ((n, ctypes.c_void_p), (n + "_token_stride", ctypes.c_int64),
                                       (n + "_head_stride", ctypes.c_int64))]


_NORM_FIELDS = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rope", ctypes.POINTER(convrot_rope_t)), ("positions", ctypes.c_void_p)]


class convrot_qk_norm_rope_t(ctypes.Structure):
    """Mirror of the C struct: one convrot_qk_norm_rope call."""
    _fields_ = [("tokens", ctypes.c_int64)] + [(f, ctypes.c_int32) for f in ("q_heads", "kv_heads", "head_dim")] + \
        _rows_fields("q", "k", "q_out", "k_out") + _NORM_FIELDS


class convrot_kv8_append_t(ctypes.Structure):
    """Mirror of the C struct: one convrot_kv8_append call."""
    _fields_ = [("cache", ctypes.POINTER(convrot_kv8_t)), ("seqs", convrot_kv8_seqs_t), ("q_heads", ctypes.c_int32)] + \
        _rows_fields("q", "k", "v", "q_out") + _NORM_FIELDS


class convrot_kv8_read_t(ctypes.Structure):
    """Mirror of the C struct: one convrot_kv8_read call."""
    _fields_ = [("cache", ctypes.POINTER(convrot_kv8_t)), ("seqs", convrot_kv8_seqs_t), ("k_out", ctypes.c_void_p),
                ("v_out", ctypes.c_void_p)]


class convrot_attn_kv8_t(ctypes.Structure):
    """Mirror of the C struct: one convrot_attn_kv8 call."""
    _fields_ = [("cache", ctypes.POINTER(convrot_kv8_t)), ("seqs", convrot_kv8_seqs_t), ("q_heads", ctypes.c_int32),
                ("causal", ctypes.c_int32)] + _rows_fields("q") + \
               [("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("scale", ctypes.c_float)]


# exported symbol -> (argtypes, restype); every name declared in convrot.h
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_WP = ctypes.POINTER(convrot_weight_t)
SIGNATURES = {
    "convrot_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "convrot_version": ([], ctypes.c_int),
    "convrot_build_id": ([], ctypes.c_char_p),
    "convrot_dynamic_group": ([_I64, _I32], _I32),
    "convrot_quantize_tensor": ([_P, _I64, _P, _P, _P], ctypes.c_int),
    "convrot_conv2d_shape": ([_P, _P, _P], ctypes.c_int),
    "convrot_conv2d_gather_plan": ([_P, _I32, _P], ctypes.c_int),
    "convrot_gemm_plan": ([_I64, _I32, _P, _P, _I32, _I32, _P], ctypes.c_int),
    "convrot_quantize_conv_weight": ([_P, _P, _WP, _P], ctypes.c_int),
    "convrot_conv2d_workspace_bytes": ([_P, _WP], _SZ),
    "convrot_conv2d_int8": ([_P, _P, _WP, _P, _P, _SZ, _P], ctypes.c_int),
    "convrot_weight4_init": ([ctypes.POINTER(convrot_weight4_t), _P, _P, _I64, _I64, _I32], ctypes.c_int),
    "convrot_quantize_weight4": ([_P, ctypes.POINTER(convrot_weight4_t), _P], ctypes.c_int),
    "convrot_linear_w4a8": ([_I64, ctypes.c_int, _P, _P, _SZ, _P], ctypes.c_int),
    "convrot_linear_w4a8_workspace_bytes": ([_I64, ctypes.c_int, _P], _SZ),
    "convrot_embed_lookup": ([_P, _I64, _P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "convrot_last_error_string": ([], ctypes.c_char_p),
    "convrot_weight_init": ([_WP, _P, _P, _I64, _I64, _I32], ctypes.c_int),
    "convrot_quantize_weight": ([_P, _WP, _P], ctypes.c_int),
    "convrot_quantize_act": ([_P, _I64, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "convrot_gemm_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "convrot_linear_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "convrot_workspace_init": ([_P, _SZ, _P], ctypes.c_int),
    "convrot_gemm_i8": ([_P, _P, _I64, _WP, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "convrot_linear_int8": ([_P, _I64, _WP, _P, _P, _SZ, _P], ctypes.c_int),
    "convrot_device_status": ([_P], ctypes.c_int),
    "convrot_linear_int8_batch": ([_I64, ctypes.c_int, ctypes.POINTER(convrot_linear_job_t), _P, _SZ, _P],
                                  ctypes.c_int),
    "convrot_linear_batch_workspace_bytes": ([_I64, ctypes.c_int, ctypes.POINTER(convrot_linear_job_t)], _SZ),
    "convrot_gemm_i8_batch": ([_I64, ctypes.c_int, ctypes.POINTER(convrot_gemm_job_t), _P, _SZ, _P], ctypes.c_int),
    "convrot_gemm_batch_workspace_bytes": ([_I64, ctypes.c_int, ctypes.POINTER(convrot_gemm_job_t)], _SZ),
    "convrot_gemm_i8_noalloc": ([_P, _P, _I64, _WP, _P, _P, _P], ctypes.c_int),
    "convrot_kv8_init": ([_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32], ctypes.c_int),
    "convrot_qk_norm_rope": ([_P, _P], ctypes.c_int),
    "convrot_kv8_append": ([_P, _P], ctypes.c_int),
    "convrot_kv8_read": ([_P, _P], ctypes.c_int),
    "convrot_attn_kv8": ([_P, _P, _SZ, _P], ctypes.c_int),
    "convrot_attn_kv8_workspace_bytes": ([_P], _SZ),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libconvrot.so.  The in-tree library is first rebuilt if it is
    missing or its build id differs from the hash of the sources beside it;
    after loading, its id must equal that hash (ImportError otherwise:
    there is no fallback path)."""
    global _lib
    if _lib is None:
        from . import build as _build
        expected = None
        if os.path.abspath(path) == os.path.abspath(LIB_PATH):
            _build.build()
            expected = _build.source_hash()
        if not os.path.exists(path):
            raise ImportError("libconvrot.so is not built (run rotated_int8_quantized_b200/build.py); "
                              "there is no fallback path")
        lib = ctypes.CDLL(path)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        if expected is not None and lib.convrot_build_id().decode() != expected:
            raise ImportError("libconvrot.so (build %s) was not built from the sources beside it (%s)"
                              % (lib.convrot_build_id().decode(), expected))
        _lib = lib
    return _lib


def build_id() -> str:
    """The loaded library's build id (hash of the sources it was built from)."""
    return load_library().convrot_build_id().decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        err = ConvrotError(status, where)
        if status == 6:
            err.args = (err.args[0] + " (" + load_library().convrot_last_error_string().decode() + ")",)
        raise err


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


@dataclass
class QuantizedWeight:
    """Rotated INT8 weight q [n, k] with FP32 row scales [n] (caller-owned
    device memory) and the C handle viewing them."""
    q: torch.Tensor
    scale: torch.Tensor
    handle: convrot_weight_t

    @property
    def n(self) -> int:
        return self.handle.n

    @property
    def k(self) -> int:
        return self.handle.k

    @property
    def group(self) -> int:
        return self.handle.group


def convrot_status_string(status: int) -> str:
    return load_library().convrot_status_string(status).decode()


def convrot_version() -> int:
    return load_library().convrot_version()


def convrot_weight_init(q: torch.Tensor, scale: torch.Tensor, group: int = GROUP) -> QuantizedWeight:
    n, k = q.shape
    h = convrot_weight_t()
    _check(load_library().convrot_weight_init(ctypes.byref(h), _ptr(q), _ptr(scale), n, k, group),
           "convrot_weight_init")
    return QuantizedWeight(q, scale, h)


def convrot_quantize_weight(w_bf16: torch.Tensor, out: QuantizedWeight, stream=None) -> QuantizedWeight:
    assert w_bf16.dtype == torch.bfloat16 and tuple(w_bf16.shape) == (out.n, out.k)
    _check(load_library().convrot_quantize_weight(_ptr(w_bf16), ctypes.byref(out.handle), _stream(stream)),
           "convrot_quantize_weight")
    return out


def convrot_quantize_act(x_bf16: torch.Tensor, xq: torch.Tensor, sx: torch.Tensor,
                         group: int = GROUP, stream=None) -> None:
    assert x_bf16.dtype == torch.bfloat16 and xq.dtype == torch.int8 and sx.dtype == torch.float32
    m, k = x_bf16.shape
    _check(load_library().convrot_quantize_act(_ptr(x_bf16), m, k, group, _ptr(xq), _ptr(sx),
                                               _stream(stream)), "convrot_quantize_act")


def convrot_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(load_library().convrot_gemm_workspace_bytes(m, n, k))


def convrot_linear_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(load_library().convrot_linear_workspace_bytes(m, n, k))


def convrot_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(load_library().convrot_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "convrot_workspace_init")


def convrot_gemm_i8(xq: torch.Tensor, sx: torch.Tensor, w: QuantizedWeight, y: Optional[torch.Tensor],
                    acc: Optional[torch.Tensor], ws: Optional[torch.Tensor], stream=None) -> None:
    m = xq.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load_library().convrot_gemm_i8(_ptr(xq), _ptr(sx), m, ctypes.byref(w.handle), _ptr(y), _ptr(acc),
                                          _ptr(ws), ws_bytes, _stream(stream)), "convrot_gemm_i8")


def convrot_linear_int8(x_bf16: torch.Tensor, w: QuantizedWeight, y: torch.Tensor, ws: torch.Tensor,
                        stream=None) -> None:
    m = x_bf16.shape[0]
    _check(load_library().convrot_linear_int8(_ptr(x_bf16), m, ctypes.byref(w.handle), _ptr(y), _ptr(ws),
                                              ws.numel() * ws.element_size(), _stream(stream)),
           "convrot_linear_int8")


def _jobs(xs, ws_, ys, biases=None):
    arr = (convrot_linear_job_t * len(xs))()
    biases = biases or [None] * len(xs)
    for i, (x, w, y, b) in enumerate(zip(xs, ws_, ys, biases)):
        arr[i].x_bf16 = _ptr(x)
        arr[i].w = ctypes.pointer(w.handle)
        arr[i].y_bf16 = _ptr(y)
        arr[i].bias_bf16 = _ptr(b)
    return arr


class LinearBatch:
    """A prepared batched call: the C job array is built once and reused,
    so a step costs one C call (argument marshalling only).  ``biases``: an
    optional BF16 [n] tensor (or None) per linear.  Linears given the same
    input tensor share its rotation."""

    def __init__(self, xs, weights, ys, ws: Optional[torch.Tensor] = None, biases=None):
        self.xs, self.weights, self.ys = list(xs), list(weights), list(ys)
        self.biases = list(biases) if biases is not None else None
        self.m = self.xs[0].shape[0]
        self.jobs = _jobs(self.xs, self.weights, self.ys, self.biases)
        need = int(load_library().convrot_linear_batch_workspace_bytes(self.m, len(self.xs), self.jobs))
        if need == 0:
            raise ConvrotError(1, "convrot_linear_batch_workspace_bytes")
        if ws is None:
            ws = torch.zeros(need, dtype=torch.uint8, device=self.xs[0].device)
        self.ws = ws

    def __call__(self, stream=None) -> None:
        _check(load_library().convrot_linear_int8_batch(self.m, len(self.xs), self.jobs, _ptr(self.ws),
                                                        self.ws.numel(), _stream(stream)),
               "convrot_linear_int8_batch")


def convrot_linear_int8_batch(xs, weights, ys, ws: torch.Tensor, stream=None, biases=None) -> None:
    """Run len(xs) linears with the same token count together."""
    m = xs[0].shape[0]
    jobs = _jobs(xs, weights, ys, biases)
    _check(load_library().convrot_linear_int8_batch(m, len(xs), jobs, _ptr(ws), ws.numel() * ws.element_size(),
                                                    _stream(stream)), "convrot_linear_int8_batch")


def convrot_linear_batch_workspace_bytes(xs, weights, ys, biases=None) -> int:
    return int(load_library().convrot_linear_batch_workspace_bytes(xs[0].shape[0], len(xs),
                                                                   _jobs(xs, weights, ys, biases)))


class GemmBatch:
    """A prepared batched GEMM call (job array built once)."""

    def __init__(self, xqs, sxs, weights, ys, accs=None, ws: Optional[torch.Tensor] = None, biases=None):
        n = len(xqs)
        accs = accs or [None] * n
        biases = biases or [None] * n
        self.keep = (list(xqs), list(sxs), list(weights), list(ys), list(accs), list(biases))
        self.m = xqs[0].shape[0]
        self.jobs = (convrot_gemm_job_t * n)()
        for i in range(n):
            self.jobs[i].xq = _ptr(xqs[i])
            self.jobs[i].sx = _ptr(sxs[i])
            self.jobs[i].w = ctypes.pointer(weights[i].handle)
            self.jobs[i].y_bf16 = _ptr(ys[i])
            self.jobs[i].acc = _ptr(accs[i])
            self.jobs[i].bias_bf16 = _ptr(biases[i])
        need = int(load_library().convrot_gemm_batch_workspace_bytes(self.m, n, self.jobs))
        if need == 0:
            raise ConvrotError(1, "convrot_gemm_batch_workspace_bytes")
        self.ws = ws if ws is not None else torch.zeros(need, dtype=torch.uint8, device=xqs[0].device)

    def __call__(self, stream=None) -> None:
        _check(load_library().convrot_gemm_i8_batch(self.m, len(self.jobs), self.jobs, _ptr(self.ws),
                                                    self.ws.numel(), _stream(stream)), "convrot_gemm_i8_batch")


def convrot_quantize_tensor(w_bf16: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None) -> None:
    """Tensor-wise simple INT8 (embedding table): q int8 like w, scale a
    one-element fp32 tensor."""
    assert w_bf16.dtype == torch.bfloat16 and q.dtype == torch.int8 and q.numel() == w_bf16.numel()
    assert scale.dtype == torch.float32 and scale.numel() == 1
    _check(load_library().convrot_quantize_tensor(_ptr(w_bf16), w_bf16.numel(), _ptr(q), _ptr(scale),
                                                  _stream(stream)), "convrot_quantize_tensor")


def convrot_embed_lookup(tokens: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor,
                         stream=None) -> None:
    """out[i] = bf16(q[tokens[i]] * scale) for int32 tokens [t], q [vocab, dim]."""
    assert tokens.dtype == torch.int32 and q.dim() == 2 and out.shape == (tokens.numel(), q.shape[1])
    _check(load_library().convrot_embed_lookup(_ptr(tokens), tokens.numel(), _ptr(q), _ptr(scale), q.shape[0],
                                               q.shape[1], _ptr(out), _stream(stream)), "convrot_embed_lookup")


# ---------------------------------------------------------------- INT4 weights (W4A8)
@dataclass
class QuantizedWeight4:
    """Packed INT4 weight q [n, k/2] (uint8) with FP32 row scales [n] and the C handle."""
    q: torch.Tensor
    scale: torch.Tensor
    handle: convrot_weight4_t

    @property
    def n(self) -> int:
        return self.handle.n

    @property
    def k(self) -> int:
        return self.handle.k

    @property
    def group(self) -> int:
        return self.handle.group


def quantize_weight4(w_bf16: torch.Tensor, stream=None, group: int = GROUP, dynamic: bool = False) -> QuantizedWeight4:
    """Offline INT4 ConvRot conversion of a BF16 weight [n, k]."""
    n, k = w_bf16.shape
    if dynamic:
        group = convrot_dynamic_group(k, group)
    q = torch.empty((n, k // 2), dtype=torch.uint8, device=w_bf16.device)
    scale = torch.empty((n,), dtype=torch.float32, device=w_bf16.device)
    h = convrot_weight4_t()
    lib = load_library()
    _check(lib.convrot_weight4_init(ctypes.byref(h), _ptr(q), _ptr(scale), n, k, group), "convrot_weight4_init")
    _check(lib.convrot_quantize_weight4(_ptr(w_bf16), ctypes.byref(h), _stream(stream)), "convrot_quantize_weight4")
    return QuantizedWeight4(q, scale, h)


class LinearBatchW4:
    """A prepared W4A8 call over up to 8 linears with the same token count."""

    def __init__(self, xs, weights, ys, ws: Optional[torch.Tensor] = None, biases=None):
        self.keep = (list(xs), list(weights), list(ys), list(biases) if biases else None)
        self.m = xs[0].shape[0]
        n = len(xs)
        biases = biases or [None] * n
        self.jobs = (convrot_linear4_job_t * n)()
        for i in range(n):
            self.jobs[i].x_bf16 = _ptr(xs[i])
            self.jobs[i].w = ctypes.pointer(weights[i].handle)
            self.jobs[i].y_bf16 = _ptr(ys[i])
            self.jobs[i].bias_bf16 = _ptr(biases[i])
        need = int(load_library().convrot_linear_w4a8_workspace_bytes(self.m, n, self.jobs))
        if need == 0:
            raise ConvrotError(3, "convrot_linear_w4a8_workspace_bytes")
        self.ws = ws if ws is not None else torch.zeros(need, dtype=torch.uint8, device=xs[0].device)

    def __call__(self, stream=None) -> None:
        _check(load_library().convrot_linear_w4a8(self.m, len(self.jobs), self.jobs, _ptr(self.ws),
                                                  self.ws.numel(), _stream(stream)), "convrot_linear_w4a8")


# ---------------------------------------------------------------- convolutions
def conv2d_geometry(x_shape, kh: int, kw: int, stride: int = 1, pad: int = 0, dilation: int = 1) -> convrot_conv2d_t:
    n, h, w, c = x_shape
    return convrot_conv2d_t(n, h, w, c, kh, kw, stride, pad, dilation)


def gemm_plan(m: int, ns, ks, w4: bool = False, sms: int = 148) -> convrot_gemm_plan_t:
    """How the GEMM kernel tiles one product (len(ns) == 1) or a batched
    launch of several (host only)."""
    count = len(ns)
    n_arr = (ctypes.c_int64 * count)(*ns)
    k_arr = (ctypes.c_int64 * count)(*ks)
    out = convrot_gemm_plan_t()
    _check(load_library().convrot_gemm_plan(m, count, n_arr, k_arr, 1 if w4 else 0, sms, ctypes.byref(out)),
           "convrot_gemm_plan")
    return out


def conv2d_gather_plan(x_shape, kh: int, kw: int, stride: int = 1, pad: int = 0, dilation: int = 1,
                       sms: int = 148) -> convrot_conv2d_plan_t:
    """The im2col gather's launch plan for a convolution (host only)."""
    g = conv2d_geometry(x_shape, kh, kw, stride, pad, dilation)
    out = convrot_conv2d_plan_t()
    _check(load_library().convrot_conv2d_gather_plan(ctypes.byref(g), sms, ctypes.byref(out)),
           "convrot_conv2d_gather_plan")
    return out


def quantize_conv_weight(w_oihw_bf16: torch.Tensor, stride: int = 1, pad: int = 0, dilation: int = 1,
                         group: Optional[int] = None, stream=None) -> QuantizedWeight:
    """Offline INT8 ConvRot conversion of a BF16 OIHW weight; the group
    defaults to the largest power of two <= 256 dividing the channels."""
    o, c, kh, kw = w_oihw_bf16.shape
    group = group or convrot_dynamic_group(c)
    k = kh * kw * c
    q = torch.empty((o, k), dtype=torch.int8, device=w_oihw_bf16.device)
    scale = torch.empty((o,), dtype=torch.float32, device=w_oihw_bf16.device)
    wt = convrot_weight_init(q, scale, group)
    g = convrot_conv2d_t(1, kh, kw, c, kh, kw, 1, 0, 1)      # only c, kh, kw matter for the weight
    _check(load_library().convrot_quantize_conv_weight(_ptr(w_oihw_bf16), ctypes.byref(g), ctypes.byref(wt.handle),
                                                       _stream(stream)), "convrot_quantize_conv_weight")
    return wt


def conv2d_int8(x_nhwc: torch.Tensor, w: QuantizedWeight, kh: int, kw: int, stride: int = 1, pad: int = 0,
                dilation: int = 1, y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """INT8 ConvRot convolution: NHWC BF16 in, NHWC BF16 out."""
    g = conv2d_geometry(x_nhwc.shape, kh, kw, stride, pad, dilation)
    lib = load_library()
    oh, ow = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.convrot_conv2d_shape(ctypes.byref(g), ctypes.byref(oh), ctypes.byref(ow)), "convrot_conv2d_shape")
    if y is None:
        y = torch.empty((g.n, oh.value, ow.value, w.n), dtype=torch.bfloat16, device=x_nhwc.device)
    if ws is None:
        need = int(lib.convrot_conv2d_workspace_bytes(ctypes.byref(g), ctypes.byref(w.handle)))
        if need == 0:
            raise ConvrotError(3, "convrot_conv2d_workspace_bytes")
        ws = torch.zeros(need, dtype=torch.uint8, device=x_nhwc.device)
    _check(lib.convrot_conv2d_int8(_ptr(x_nhwc), ctypes.byref(g), ctypes.byref(w.handle), _ptr(y), _ptr(ws),
                                   ws.numel(), _stream(stream)), "convrot_conv2d_int8")
    return y


# ---------------------------------------------------------------- attention beside the linears
def rope_table(positions: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """FP32 [positions, rot_dim / 2, 2] cosines and sines of position *
    theta^(-2 i / rot_dim), the angles taken in 64 bits."""
    inv = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(device)


@dataclass
class Rope:
    """The position rotation: cos_sin fp32 [positions, rot_dim / 2, 2]
    (rope_table), adjacent pairs (2 i, 2 i + 1) or pairs (i, i + rot_dim / 2),
    and for several position axes a uint8 [rot_dim / 2] naming each pair's."""
    cos_sin: torch.Tensor
    adjacent: bool = False
    axis: Optional[torch.Tensor] = None


class KV8Cache:
    """A paged INT8 key/value cache over caller-owned tensors: k, v int8
    [pages, kv_heads, page_tokens, head_dim]; k_scale, v_scale fp32
    [pages, kv_heads, page_tokens / 16]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        pages, heads, page, dim = k.shape
        scales = (pages, heads, page // 16)
        if v.shape != k.shape or tuple(k_scale.shape) != scales or tuple(v_scale.shape) != scales:
            raise ValueError("expected codes [pages, kv_heads, page_tokens, head_dim] and scales "
                             "[pages, kv_heads, page_tokens / 16]")
        _want(torch.int8, k=k, v=v)
        _want(torch.float32, k_scale=k_scale, v_scale=v_scale)
        _one_device(k, v, k_scale, v_scale)
        self.handle = convrot_kv8_t()
        _check(load_library().convrot_kv8_init(ctypes.byref(self.handle), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                                               pages, heads, page, dim), "convrot_kv8_init")


def make_kv8_cache(pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda") -> KV8Cache:
    """Allocate a cache (nothing in it is read before a call has stored it)."""
    codes = [torch.empty((pages, kv_heads, page_tokens, head_dim), dtype=torch.int8, device=device) for _ in "kv"]
    scales = [torch.empty((pages, kv_heads, page_tokens // 16), dtype=torch.float32, device=device) for _ in "kv"]
    return KV8Cache(*codes, *scales)


def _want(dtype, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.dtype != dtype:
            raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))


def _one_device(*tensors) -> torch.device:
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1:
        raise ValueError("tensors on several devices: %s" % sorted(map(str, devices)))
    return devices.pop()


def _set_rows(job, name: str, t: Optional[torch.Tensor], heads: int, dim: int, tokens: int) -> None:
    """A [tokens, heads, dim] BF16 view into a job's pointer and strides."""
    if t is None:
        return
    if t.dtype != torch.bfloat16 or tuple(t.shape) != (tokens, heads, dim):
        raise ValueError("%s: expected BF16 [%d, %d, %d], got %s %s" % (name, tokens, heads, dim, t.dtype, tuple(t.shape)))
    if not t.is_cuda or t.stride(2) != 1:
        raise ValueError("%s: expected a CUDA tensor whose rows are contiguous" % name)
    setattr(job, name, t.data_ptr())
    # the stride of a single token or head means nothing
    setattr(job, name + "_token_stride", t.stride(0) if tokens > 1 else 0)
    setattr(job, name + "_head_stride", t.stride(1) if heads > 1 else 0)


def _set_seqs(s: convrot_kv8_seqs_t, tokens: int, table: torch.Tensor, kv_len: torch.Tensor,
              cu: Optional[torch.Tensor]) -> None:
    _want(torch.int32, page_table=table, kv_len=kv_len, cu=cu)
    if table.dim() != 2 or tuple(kv_len.shape) != (table.shape[0],) or \
            (cu is not None and tuple(cu.shape) != (table.shape[0] + 1,)):
        raise ValueError("expected page_table [batch, max_pages], kv_len [batch] and cu [batch + 1]")
    s.page_table, s.kv_len, s.cu = _ptr(table), _ptr(kv_len), _ptr(cu)
    s.tokens, s.batch, s.max_pages = tokens, table.shape[0], table.shape[1]


def _set_norm(job, dim, tokens, q_weight, k_weight, eps, rope: Optional[Rope], positions) -> list:
    """Fills in weights and rotation; returns what has to stay alive."""
    _want(torch.bfloat16, q_weight=q_weight, k_weight=k_weight)
    for w in (q_weight, k_weight):
        if w is not None and tuple(w.shape) != (dim,):
            raise ValueError("expected norm weights [%d], got %s" % (dim, tuple(w.shape)))
    job.q_weight, job.k_weight, job.eps = _ptr(q_weight), _ptr(k_weight), eps
    if rope is None:
        return [q_weight, k_weight]
    table, axes = rope.cos_sin, 1
    _want(torch.float32, cos_sin=table)
    _want(torch.uint8, axis=rope.axis)
    if table.dim() != 3 or table.shape[2] != 2 or (rope.axis is not None and tuple(rope.axis.shape) != (table.shape[1],)):
        raise ValueError("expected cos_sin [positions, rot_dim / 2, 2] and axis [rot_dim / 2]")
    if positions is not None:
        _want(torch.int32, positions=positions)
        if positions.shape[-1] != tokens or positions.dim() not in (1, 2):
            raise ValueError("expected positions [tokens] or [axes, tokens]")
        axes = positions.shape[0] if positions.dim() == 2 else 1
    r = convrot_rope_t(_ptr(table), table.shape[0], 2 * table.shape[1], 1 if rope.adjacent else 0, _ptr(rope.axis), axes)
    job.rope, job.positions = ctypes.pointer(r), _ptr(positions)
    return [q_weight, k_weight, rope, positions, r]


class _Prepared:
    """A prepared call: its C struct is built once, a step costs one C call
    on the tensors' own device.  The tensors stay the caller's: new values
    in them are what the next call works on."""
    _entry = ""
    _cleared = None                       # event behind the clearing of a workspace that the call made itself,
    _behind: set = frozenset()            # and the streams whose work is ordered behind it

    def _prepare(self, job, device: torch.device, *more) -> None:
        self.device = device
        self._call = getattr(load_library(), self._entry)
        self._args = (ctypes.byref(job),) + more

    def __call__(self, stream=None) -> None:
        index = self.device.index
        if torch.cuda.current_device() != index:
            with torch.cuda.device(self.device):
                return self(stream)
        if stream is None:
            # the current stream's handle without the Stream object around it (a microsecond of a small call's eight)
            handle = torch._C._cuda_getCurrentRawStream(index)
        else:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if self._cleared is not None and handle not in self._behind:
            self._wait_for_clear(handle)
        status = self._call(*self._args, handle)
        if status:
            _check(status, self._entry)


class QKNormRope(_Prepared):
    """Norm and rotation of q [tokens, q_heads, head_dim] and (or None) k
    [tokens, kv_heads, head_dim] into q_out, k_out (they may be q and k)."""
    _entry = "convrot_qk_norm_rope"

    def __init__(self, q, k, q_out, k_out, q_weight=None, k_weight=None, eps: float = 1e-6, rope: Optional[Rope] = None,
                 positions=None):
        tokens, heads, dim = q.shape
        j = self.job = convrot_qk_norm_rope_t()
        j.tokens, j.q_heads, j.kv_heads, j.head_dim = tokens, heads, 0 if k is None else k.shape[1], dim
        for name, t, h in (("q", q, heads), ("k", k, j.kv_heads), ("q_out", q_out, heads), ("k_out", k_out, j.kv_heads)):
            _set_rows(j, name, t, h, dim, tokens)
        self.keep = [q, k, q_out, k_out, _set_norm(j, dim, tokens, q_weight, k_weight, eps, rope, positions)]
        self._prepare(j, _one_device(q, k, q_out, k_out, q_weight, k_weight, positions,
                                     *([rope.cos_sin, rope.axis] if rope else [])))


class KV8Append(_Prepared):
    """Append a step's k, v [tokens, kv_heads, head_dim] to the cache, k
    normalised and rotated, and put q (or None), normalised and rotated,
    into q_out.  kv_len counts the new tokens; cu None: one per sequence;
    positions None: the position in the sequence."""
    _entry = "convrot_kv8_append"

    def __init__(self, q, k, v, cache: KV8Cache, page_table, kv_len, q_out=None, cu=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, rope: Optional[Rope] = None, positions=None):
        h = cache.handle
        tokens = k.shape[0]
        j = self.job = convrot_kv8_append_t()
        j.cache, j.q_heads = ctypes.pointer(h), 0 if q is None else q.shape[1]
        _set_seqs(j.seqs, tokens, page_table, kv_len, cu)
        for name, t, n in (("q", q, j.q_heads), ("k", k, h.kv_heads), ("v", v, h.kv_heads), ("q_out", q_out, j.q_heads)):
            _set_rows(j, name, t, n, h.head_dim, tokens)
        self.keep = [q, k, v, q_out, cache, page_table, kv_len, cu,
                     _set_norm(j, h.head_dim, tokens, q_weight, k_weight, eps, rope, positions)]
        self._prepare(j, _one_device(q, k, v, q_out, cache.k, page_table, kv_len, cu, q_weight, k_weight, positions,
                                     *([rope.cos_sin, rope.axis] if rope else [])))


class KV8Read(_Prepared):
    """The last cu[b + 1] - cu[b] cached tokens of every sequence as BF16
    rows of k_out and v_out [tokens, kv_heads, head_dim] (one may be None)."""
    _entry = "convrot_kv8_read"

    def __init__(self, cache: KV8Cache, page_table, kv_len, k_out, v_out, cu=None):
        h = cache.handle
        if k_out is None and v_out is None:
            raise ValueError("expected k_out, v_out or both")
        tokens = (k_out if k_out is not None else v_out).shape[0]
        j = self.job = convrot_kv8_read_t()
        j.cache = ctypes.pointer(h)
        _set_seqs(j.seqs, tokens, page_table, kv_len, cu)
        for t in (k_out, v_out):
            if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != (tokens, h.kv_heads, h.head_dim)):
                raise ValueError("expected BF16 outputs [%d, %d, %d]" % (tokens, h.kv_heads, h.head_dim))
        j.k_out, j.v_out = _ptr(k_out), _ptr(v_out)
        self.keep = [cache, page_table, kv_len, k_out, v_out, cu]
        self._prepare(j, _one_device(cache.k, page_table, kv_len, k_out, v_out, cu))


class AttnKV8(_Prepared):
    """Attention of q [tokens, q_heads, head_dim] over the cache into out
    (contiguous, BF16) and, if given, lse [tokens, q_heads] (fp32).  The
    rows of sequence b are its last cu[b + 1] - cu[b] tokens; without
    `causal` every one of them sees all kv_len[b].  ws: a
    workspace of at least `ws_bytes`, zero-filled before its first call
    (allocated here if None); AttnKV8 calls of any shapes may share one, but
    neither calls that run at the same time nor the linears' calls."""
    _entry = "convrot_attn_kv8"

    def __init__(self, q, cache: KV8Cache, page_table, kv_len, out, cu=None, lse=None, scale: Optional[float] = None,
                 causal: bool = True, ws: Optional[torch.Tensor] = None):
        h = cache.handle
        tokens, heads, dim = q.shape
        j = self.job = convrot_attn_kv8_t()
        j.cache, j.q_heads, j.causal = ctypes.pointer(h), heads, 1 if causal else 0
        j.scale = dim ** -0.5 if scale is None else scale
        _set_seqs(j.seqs, tokens, page_table, kv_len, cu)
        _set_rows(j, "q", q, heads, h.head_dim, tokens)
        if out.dtype != torch.bfloat16 or tuple(out.shape) != tuple(q.shape):
            raise ValueError("out: expected BF16 %s" % (tuple(q.shape),))
        _want(torch.float32, lse=lse)
        if lse is not None and tuple(lse.shape) != (tokens, heads):
            raise ValueError("lse: expected [%d, %d]" % (tokens, heads))
        j.out, j.lse = _ptr(out), _ptr(lse)
        device = _one_device(q, cache.k, page_table, kv_len, out, cu, lse, ws)
        with torch.cuda.device(device):
            self.ws_bytes = int(load_library().convrot_attn_kv8_workspace_bytes(ctypes.byref(j)))
        if ws is None:
            # an invalid job needs none: the call says what is wrong with it
            with torch.cuda.device(device):
                ws = torch.zeros(max(self.ws_bytes, 256), dtype=torch.uint8, device=device)
                if not torch.cuda.is_current_stream_capturing():             # a graph clears it in its own order
                    self._cleared = torch.cuda.Event()
                    self._cleared.record()
                    self._behind = {torch._C._cuda_getCurrentRawStream(device.index)}
        self.ws = ws
        self.keep = [q, cache, page_table, kv_len, out, cu, lse]
        self._prepare(j, device, _ptr(ws), ws.numel() * ws.element_size())

    def _wait_for_clear(self, handle: int) -> None:
        """Another stream's first call waits until the workspace made here is
        cleared.  A stream that is being captured cannot wait for work outside
        its graph: torch.cuda.graph has synchronised the device before."""
        with _allocating(handle, self.device):
            if torch.cuda.is_current_stream_capturing():
                return
            side = torch.cuda.current_stream()
            side.wait_event(self._cleared)
            self.ws.record_stream(side)
        self._behind.add(handle)


def _allocating(stream, device):
    """Where the functions below make their tensors: on the stream they
    launch on, so that fills and frees are ordered with the kernels."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), device)
    return torch.cuda.stream(stream)


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, eps: float = 1e-6, rope: Optional[Rope] = None, positions=None,
                 stream=None):
    """QKNormRope into new tensors; returns (q_out, k_out)."""
    with _allocating(stream, q.device):
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    QKNormRope(q, k, q_out, k_out, q_weight, k_weight, eps, rope, positions)(stream)
    return q_out, k_out


def kv8_append(q, k, v, cache: KV8Cache, page_table, kv_len, cu=None, q_weight=None, k_weight=None, eps: float = 1e-6,
               rope: Optional[Rope] = None, positions=None, stream=None):
    """KV8Append with a new q_out, which it returns (None without q; rows
    behind the last sequence hold anything)."""
    with _allocating(stream, k.device):
        q_out = None if q is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    KV8Append(q, k, v, cache, page_table, kv_len, q_out, cu, q_weight, k_weight, eps, rope, positions)(stream)
    return q_out


def kv8_read(cache: KV8Cache, page_table, kv_len, tokens: Optional[int] = None, cu=None, stream=None):
    """KV8Read into new tensors of `tokens` rows (batch rows without cu)."""
    if cu is not None and tokens is None:
        raise ValueError("tokens: with cu the number of rows has to be given")
    shape = (tokens if cu is not None else page_table.shape[0], cache.handle.kv_heads, cache.handle.head_dim)
    with _allocating(stream, cache.k.device):
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=cache.k.device) for _ in "kv")
    KV8Read(cache, page_table, kv_len, k, v, cu)(stream)
    return k, v


def attn_kv8(q, cache: KV8Cache, page_table, kv_len, cu=None, scale: Optional[float] = None, causal: bool = True, ws=None,
             stream=None):
    """AttnKV8 into new tensors; returns (out, lse)."""
    with _allocating(stream, q.device):
        out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=q.device)
        call = AttnKV8(q, cache, page_table, kv_len, out, cu, lse, scale, causal, ws)
    call(stream)
    return out, lse


def convrot_device_status(stream=None) -> None:
    _check(load_library().convrot_device_status(_stream(stream)), "convrot_device_status")


# ---------------------------------------------------------------- helpers
def convrot_dynamic_group(k: int, max_group: int = GROUP) -> int:
    """The group --dynamic-convrot picks for k input features (0: none)."""
    return int(load_library().convrot_dynamic_group(k, max_group))


def quantize_weight(w_bf16: torch.Tensor, stream=None, group: int = GROUP, dynamic: bool = False) -> QuantizedWeight:
    """Allocate q/scale and run the offline rotate+quantise kernel; with
    dynamic=True the group is the largest power of two <= group dividing k."""
    n, k = w_bf16.shape
    if dynamic:
        group = convrot_dynamic_group(k, group)
    q = torch.empty((n, k), dtype=torch.int8, device=w_bf16.device)
    scale = torch.empty((n,), dtype=torch.float32, device=w_bf16.device)
    return convrot_quantize_weight(w_bf16, convrot_weight_init(q, scale, group), stream)


def make_workspace(m: int, w: QuantizedWeight, device=None, linear: bool = True) -> torch.Tensor:
    """A zero-filled workspace big enough for convrot_linear_int8 (or, with
    linear=False, convrot_gemm_i8) at m rows against w."""
    nbytes = (convrot_linear_workspace_bytes if linear else convrot_gemm_workspace_bytes)(m, w.n, w.k)
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device or w.q.device)


def linear_int8(x_bf16: torch.Tensor, w: QuantizedWeight, ws: torch.Tensor, y: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty((x_bf16.shape[0], w.n), dtype=torch.bfloat16, device=x_bf16.device)
    convrot_linear_int8(x_bf16, w, y, ws, stream)
    return y
