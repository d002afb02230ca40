"""GB300-native MLP training step: CUDA kernels for sm_103a behind a C ABI.

This module is the thin Python binding of ``libmlp_step.so`` (declared in
``include/mlp_step.h``).  It only marshals arguments: tensors become device
pointers, the current torch CUDA stream becomes the ``cudaStream_t``, and a
non-zero status becomes :class:`MlpError`.  Every step of the computation runs
in the library's kernels; if the library is missing, calls raise instead of
falling back to anything else.

PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "MlpError", "load", "lib_path",
    "MLP_ACT_NONE", "MLP_ACT_RELU", "MLP_ACT_LEAKY_RELU_SQ", "MLP_ACT_GELU",
    "MLP_ACT_GELU_TANH", "MLP_ACT_SILU", "MLP_CKPT8_GROUP",
    "MLP_PREC_FP32", "MLP_PREC_BF16", "MLP_PREC_FP16", "MLP_DTYPE_F32", "MLP_DTYPE_BF16",
    "MLP_DTYPE_U8", "MLP_DTYPE_F16", "MLP_ORDER_FAST", "MLP_ORDER_LINEAR",
]

MLP_OK = 0
MLP_ERR_INVALID_ARG = 1
MLP_ERR_MISALIGNED = 2
MLP_ERR_UNSUPPORTED_SHAPE = 3
MLP_ERR_CUDA = 4
MLP_ERR_DEVICE_TIMEOUT = 5
MLP_ERR_NUMERIC = 6

MLP_ACT_NONE = 0
MLP_ACT_RELU = 1
MLP_ACT_LEAKY_RELU_SQ = 2
MLP_ACT_GELU = 3
MLP_ACT_GELU_TANH = 4
MLP_ACT_SILU = 5
MLP_PREC_FP32 = 0
MLP_PREC_BF16 = 1
MLP_PREC_FP16 = 2
MLP_DTYPE_F32 = 0
MLP_DTYPE_BF16 = 1
MLP_DTYPE_U8 = 2
MLP_DTYPE_F16 = 3
MLP_ORDER_FAST = 0
MLP_ORDER_LINEAR = 1
MLP_CKPT8_GROUP = 32

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libmlp_step.so")
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong

# name -> (restype, argtypes); the signatures of include/mlp_step.h
SIGNATURES = {
    "mlp_status_string": (ctypes.c_char_p, [_i]),
    "mlp_get_device_status": (_i, [_vp]),
    "mlp_set_wait_limit_ns": (None, [_ll]),
    "mlp_set_reduction_order": (_i, [_i]),
    "mlp_attn_prep_fwd": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, ctypes.c_float,
                               ctypes.c_float, _vp, _vp, _vp]),
    "mlp_get_reduction_order": (_i, []),
    "mlp_selftest_wait_timeout": (_i, [_ll, _vp]),
    "mlp_launch_count": (ctypes.c_ulonglong, []),
    "mlp_timing_enable": (_i, [_i]),
    "mlp_timing_report": (_sz, [ctypes.c_char_p, _sz]),
    "mlp_param_count": (_sz, [_vp, _i]),
    "mlp_param_offset": (_sz, [_vp, _i, _i, _i]),
    "mlp_shadow_elems": (_sz, [_vp, _i]),
    "mlp_workspace_bytes": (_sz, [_vp, _i, _i, _i]),
    "mlp_create": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, ctypes.POINTER(_vp)]),
    "mlp_destroy": (None, [_vp]),
    "mlp_refresh_shadow": (_i, [_vp, _vp]),
    "mlp_forward": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "mlp_backward": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "mlp_sgd_step": (_i, [_vp, _f, _f, _vp]),
    "mlp_train_step": (_i, [_vp, _vp, _i, _vp, _i, _f, _f, _vp, _vp, _vp]),
    "mlp_train_epoch": (_i, [_vp, _vp, _i, _vp, _i, _i, _f, _f, _vp, _vp, _vp]),
    "softmax_xent_workspace_bytes": (_sz, [_i, _i]),
    "softmax_xent_fwd_bwd": (_i, [_vp, _i, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp]),
    "softmax_xent_noalloc_max_batch": (_i, []),
    "softmax_xent_fwd_bwd_noalloc": (_i, [_vp, _i, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp]),
    "sgd_momentum_step": (_i, [_vp, _vp, _vp, _vp, _sz, _f, _f, _vp]),
    "mlp_gemm": (_i, [_i, _i, _i, _vp, _i, _i, _vp, _i, _i, _i, _vp, _i, _vp, _i, _vp, _i, _i,
                      _vp]),
    "mlp_colsum_workspace_bytes": (_sz, [_i, _i]),
    "mlp_colsum": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "mlp_block_workspace_bytes": (_sz, [_i, _i, _i]),
    "mlp_block_fwd": (_i, [_vp, _vp, _vp, _i, _i, _i, _f, _f, _vp, _vp, _vp]),
    "mlp_block_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _sz,
                           _vp]),
    "mse_workspace_bytes": (_sz, [_sz]),
    "mse_loss_fwd_bwd": (_i, [_vp, _vp, _sz, _vp, _vp, _vp, _sz, _vp]),
    "mlp_stack_param_count": (_sz, [_i, _i, _i]),
    "mlp_stack_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "mlp_stack_train_step": (_i, [_i, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _f, _f,
                                  _vp, _vp, _sz, _vp]),
    "mlp_ckpt8_scale_cols": (_i, [_i]),
    "mlp_ckpt8_encode": (_i, [_vp, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp]),
    "mlp_ckpt8_decode": (_i, [_vp, _i, _vp, _i, _i, _i, _vp, _i, _i, _vp]),
    "mlp_stack_ckpt8_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "mlp_stack_train_step_ckpt8": (_i, [_i, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _f,
                                        _f, _vp, _vp, _sz, _vp]),
    "mlp_layernorm_fwd": (_i, [_vp, _i, _i, _vp, _vp, _i, _i, _f, _vp, _i, _vp, _vp, _vp, _i,
                               _vp, _i, _vp]),
    "mlp_layernorm_workspace_bytes": (_sz, [_i, _i]),
    "mlp_layernorm_bwd": (_i, [_vp, _i, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i,
                               _i, _i, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "mlp_linear_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "mlp_linear_fwd": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _i, _f, _vp, _i, _vp, _i, _i,
                            _vp, _i, _vp, _i, _vp, _i, _vp, _sz, _vp]),
    "mlp_linear_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "mlp_linear_bwd": (_i, [_vp, _i, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _i, _vp, _i,
                            _vp, _i, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "mlp_act_bwd_workspace_bytes": (_sz, [_i, _i]),
    "mlp_act_bwd": (_i, [_vp, _i, _i, _i, _i, _i, _f, _vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp,
                         _vp, _i, _vp, _sz, _vp]),
}


class MlpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = load().mlp_status_string(status).decode() if _lib is not None else str(status)
        super().__init__("%s: %s (status %d)" % (where, msg, status))


def load():
    """Loads libmlp_step.so (built by ``mlp_step_gb300.build``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise ImportError("libmlp_step.so is not built; run mlp_step_gb300.build.build()")
        lib = ctypes.CDLL(lib_path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


# ------------------------------------------------------------------ helpers

def _ptr(t):
    """Device address of a tensor the library reads as row-major rows: the
    last dimension must be unit-stride (rows may be padded, their pitch is
    passed as the leading dimension), and tensors of more than two
    dimensions must be contiguous."""
    if t is None:
        return None
    if t.dim() >= 1 and t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError("the library reads row-major rows: last dimension must have stride 1 "
                         "(got strides %s)" % (tuple(t.stride()),))
    if t.dim() > 2 and not t.is_contiguous():
        raise ValueError("tensors of more than two dimensions must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, where):
    if status != MLP_OK:
        raise MlpError(status, where)


def _dims(dims):
    return (ctypes.c_int * len(dims))(*dims), len(dims)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return MLP_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return MLP_DTYPE_BF16
    if t.dtype == torch.uint8:
        return MLP_DTYPE_U8
    if t.dtype == torch.float16:
        return MLP_DTYPE_F16
    raise TypeError("unsupported dtype %s" % t.dtype)


# ------------------------------------------------------------------ status

def status_string(s: int) -> str:
    return load().mlp_status_string(s).decode()


def get_device_status(stream=None) -> int:
    return load().mlp_get_device_status(_stream(stream))


def set_wait_limit_ns(ns: int) -> None:
    load().mlp_set_wait_limit_ns(int(ns))


def set_reduction_order(order: int) -> None:
    """MLP_ORDER_FAST or MLP_ORDER_LINEAR (see mlp_step.h)."""
    _check(load().mlp_set_reduction_order(int(order)), "mlp_set_reduction_order")


def get_reduction_order() -> int:
    return load().mlp_get_reduction_order()


def selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(load().mlp_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "mlp_selftest_wait_timeout")


def launch_count() -> int:
    """Kernels enqueued (or captured) by the library since it was loaded."""
    return load().mlp_launch_count()


def timing_enable(on: bool) -> None:
    load().mlp_timing_enable(1 if on else 0)


def timing_report() -> dict:
    """{"kernel[shape]": (launches, total_ms)} for launches since timing_enable(True)."""
    import json
    L = load()
    need = L.mlp_timing_report(None, 0)
    buf = ctypes.create_string_buffer(need + 16)
    L.mlp_timing_report(buf, len(buf))
    return {k: (v[0], v[1]) for k, v in json.loads(buf.value.decode()).items()}


# ------------------------------------------------------------------ MLP

def mlp_param_count(dims) -> int:
    d, n = _dims(dims)
    return load().mlp_param_count(d, n)


def mlp_param_offset(dims, layer: int, which: int) -> int:
    d, n = _dims(dims)
    return load().mlp_param_offset(d, n, layer, which)


def mlp_shadow_elems(dims) -> int:
    d, n = _dims(dims)
    return load().mlp_shadow_elems(d, n)


def mlp_workspace_bytes(dims, max_batch: int, prec: int) -> int:
    d, n = _dims(dims)
    return load().mlp_workspace_bytes(d, n, max_batch, prec)


class MLP:
    """Owner of the device buffers of one MLP (flat params, velocity, grads,
    the 16-bit weight shadow of the tensor-core precisions, workspace) and of
    the library handle over them."""

    def __init__(self, dims, prec=MLP_PREC_BF16, max_batch=128, params=None,
                 hidden_act=MLP_ACT_RELU, device="cuda"):
        import torch
        self.dims = list(dims)
        self.prec = prec
        self.max_batch = max_batch
        n = mlp_param_count(self.dims)
        self.params = torch.zeros(n, dtype=torch.float32, device=device)
        if params is not None:
            self.params.copy_(torch.as_tensor(params, dtype=torch.float32))
        self.velocity = torch.zeros_like(self.params)
        self.grads = torch.zeros_like(self.params)
        self.shadow = None
        if prec in (MLP_PREC_BF16, MLP_PREC_FP16):
            self.shadow = torch.zeros(mlp_shadow_elems(self.dims),
                                      dtype=torch.bfloat16 if prec == MLP_PREC_BF16
                                      else torch.float16, device=device)
        wsb = mlp_workspace_bytes(self.dims, max_batch, prec)
        self.workspace = torch.empty(wsb, dtype=torch.uint8, device=device)
        d, nd = _dims(self.dims)
        h = ctypes.c_void_p()
        _check(load().mlp_create(d, nd, hidden_act, prec, max_batch, _ptr(self.params),
                                 _ptr(self.velocity), _ptr(self.grads), _ptr(self.shadow),
                                 _ptr(self.workspace), wsb, ctypes.byref(h)), "mlp_create")
        self.handle = h
        self.refresh_shadow()

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.mlp_destroy(self.handle)
            self.handle = None

    def refresh_shadow(self, stream=None):
        _check(load().mlp_refresh_shadow(self.handle, _stream(stream)), "mlp_refresh_shadow")

    def forward(self, x, logits, stream=None):
        _check(load().mlp_forward(self.handle, _ptr(x), _dtype_code(x), x.shape[0], _ptr(logits),
                                  _stream(stream)), "mlp_forward")

    def backward(self, dlogits, batch, dx=None, stream=None):
        _check(load().mlp_backward(self.handle, _ptr(dlogits), dlogits.shape[1], batch, _ptr(dx),
                                   _stream(stream)), "mlp_backward")

    def sgd_step(self, lr, momentum, stream=None):
        _check(load().mlp_sgd_step(self.handle, lr, momentum, _stream(stream)), "mlp_sgd_step")

    def train_step(self, x, labels, lr, momentum, loss_out=None, argmax_out=None, batch=None,
                   stream=None):
        b = x.shape[0] if batch is None else batch
        _check(load().mlp_train_step(self.handle, _ptr(x), _dtype_code(x), _ptr(labels), b, lr,
                                     momentum, _ptr(loss_out), _ptr(argmax_out),
                                     _stream(stream)), "mlp_train_step")

    def train_epoch(self, x, labels, lr, momentum, batch, losses_out=None, argmax_out=None,
                    n_samples=None, stream=None):
        """Training steps over x / labels in order, `batch` rows at a time (the
        last step takes the remainder); losses_out: fp32[n_steps]."""
        n = x.shape[0] if n_samples is None else n_samples
        _check(load().mlp_train_epoch(self.handle, _ptr(x), _dtype_code(x), _ptr(labels), n,
                                      batch, lr, momentum, _ptr(losses_out), _ptr(argmax_out),
                                      _stream(stream)), "mlp_train_epoch")


# ------------------------------------------------------------------ single kernels

def softmax_xent_workspace_bytes(batch: int, classes: int) -> int:
    return load().softmax_xent_workspace_bytes(batch, classes)


def softmax_xent_fwd_bwd(logits, labels, loss_out, dlogits=None, argmax_out=None,
                         workspace=None, classes=None, stream=None):
    B = logits.shape[0]
    C = logits.shape[1] if classes is None else classes
    dl_dtype = _dtype_code(dlogits) if dlogits is not None else MLP_DTYPE_F32
    ldd = dlogits.shape[1] if dlogits is not None else C
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().softmax_xent_fwd_bwd(_ptr(logits), logits.stride(0), _ptr(labels), B, C,
                                       _ptr(loss_out), _ptr(dlogits), dl_dtype, ldd,
                                       _ptr(argmax_out), _ptr(workspace), wsb, _stream(stream)),
           "softmax_xent_fwd_bwd")


def softmax_xent_fwd_bwd_noalloc(logits, labels, loss_out, dlogits=None, argmax_out=None,
                                 classes=None, stream=None):
    """softmax_xent_fwd_bwd with the library's fixed device scratch (no workspace)."""
    B = logits.shape[0]
    C = logits.shape[1] if classes is None else classes
    dl_dtype = _dtype_code(dlogits) if dlogits is not None else MLP_DTYPE_F32
    ldd = dlogits.shape[1] if dlogits is not None else C
    _check(load().softmax_xent_fwd_bwd_noalloc(_ptr(logits), logits.stride(0), _ptr(labels), B,
                                               C, _ptr(loss_out), _ptr(dlogits), dl_dtype, ldd,
                                               _ptr(argmax_out), _stream(stream)),
           "softmax_xent_fwd_bwd_noalloc")


def sgd_momentum_step(w, g, v, lr, momentum, w_bf16=None, stream=None):
    _check(load().sgd_momentum_step(_ptr(w), _ptr(g), _ptr(v), _ptr(w_bf16), w.numel(), lr,
                                    momentum, _stream(stream)), "sgd_momentum_step")


def mlp_gemm(A, B, C, M, N, K, a_trans=False, b_trans=False, bias=None, act=MLP_ACT_NONE,
             mask=None, stream=None):
    """C = epilogue(op(A) @ op(B)); tensors are 2-D row-major with unit inner stride."""
    in_dtype = _dtype_code(A)
    _check(load().mlp_gemm(M, N, K, _ptr(A), A.stride(0), int(a_trans), _ptr(B), B.stride(0),
                           int(b_trans), in_dtype, _ptr(bias), act, _ptr(mask),
                           mask.stride(0) if mask is not None else 0, _ptr(C), C.stride(0),
                           _dtype_code(C), _stream(stream)), "mlp_gemm")


def mlp_colsum_workspace_bytes(rows: int, cols: int) -> int:
    return load().mlp_colsum_workspace_bytes(rows, cols)


def mlp_colsum(X, out, rows=None, cols=None, workspace=None, stream=None):
    r = X.shape[0] if rows is None else rows
    c = out.shape[0] if cols is None else cols
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().mlp_colsum(_ptr(X), _dtype_code(X), r, c, X.stride(0), _ptr(out),
                             _ptr(workspace), wsb, _stream(stream)), "mlp_colsum")


def mse_workspace_bytes(n: int) -> int:
    return load().mse_workspace_bytes(n)


def mse_loss_fwd_bwd(y, t, loss_out, dy, workspace, stream=None):
    wsb = workspace.numel() * workspace.element_size()
    _check(load().mse_loss_fwd_bwd(_ptr(y), _ptr(t), y.numel(), _ptr(loss_out), _ptr(dy),
                                   _ptr(workspace), wsb, _stream(stream)), "mse_loss_fwd_bwd")


# ------------------------------------------------------------------ block

def mlp_block_workspace_bytes(T: int, d: int, hidden: int) -> int:
    return load().mlp_block_workspace_bytes(T, d, hidden)


def mlp_block_fwd(x, w_gate, w_down, y, rstd, eps=1e-6, slope=0.5, stream=None):
    T, d = x.shape
    h = w_gate.shape[1]
    _check(load().mlp_block_fwd(_ptr(x), _ptr(w_gate), _ptr(w_down), T, d, h, eps, slope,
                                _ptr(y), _ptr(rstd), _stream(stream)), "mlp_block_fwd")


def mlp_block_bwd(x, rstd, w_gate, w_down, dy, dx, dw_gate, dw_down, workspace, eps=1e-6,
                  slope=0.5, stream=None):
    T, d = x.shape
    h = w_gate.shape[1]
    wsb = workspace.numel() * workspace.element_size()
    _check(load().mlp_block_bwd(_ptr(x), _ptr(rstd), _ptr(w_gate), _ptr(w_down), _ptr(dy), T, d,
                                h, eps, slope, _ptr(dx), _ptr(dw_gate), _ptr(dw_down),
                                _ptr(workspace), wsb, _stream(stream)), "mlp_block_bwd")


def mlp_attn_prep_fwd(x, w_qkv, q_gain, qkv_out, rstd_out, n_q_heads, n_kv_heads,
                      rope_dims, seq_len, eps=1e-6, rope_theta=10000.0, head_dim=64, stream=None):
    """Fused RMSNorm -> QKV projection -> QK norm -> partial RoPE -> q gain."""
    T, d = x.shape
    _check(load().mlp_attn_prep_fwd(_ptr(x), _ptr(w_qkv), _ptr(q_gain), T, d, n_q_heads,
                                    n_kv_heads, head_dim, rope_dims, seq_len, eps, rope_theta,
                                    _ptr(qkv_out), _ptr(rstd_out), _stream(stream)),
           "mlp_attn_prep_fwd")


def mlp_stack_param_count(n_blocks: int, d: int, hidden: int) -> int:
    return load().mlp_stack_param_count(n_blocks, d, hidden)


def mlp_stack_workspace_bytes(n_blocks: int, T: int, d: int, hidden: int) -> int:
    return load().mlp_stack_workspace_bytes(n_blocks, T, d, hidden)


def mlp_stack_train_step(n_blocks, T, d, hidden, x0, target, params, velocity, grads,
                         params_bf16, lr, momentum, loss_out, workspace, eps=1e-6, slope=0.5,
                         stream=None):
    wsb = workspace.numel() * workspace.element_size()
    _check(load().mlp_stack_train_step(n_blocks, T, d, hidden, eps, slope, _ptr(x0), _ptr(target),
                                       _ptr(params), _ptr(velocity), _ptr(grads),
                                       _ptr(params_bf16), lr, momentum, _ptr(loss_out),
                                       _ptr(workspace), wsb, _stream(stream)),
           "mlp_stack_train_step")


def mlp_stack_ckpt8_workspace_bytes(n_blocks: int, T: int, d: int, hidden: int) -> int:
    return load().mlp_stack_ckpt8_workspace_bytes(*_sizes(n_blocks, T, d, hidden))


def mlp_stack_train_step_ckpt8(n_blocks, T, d, hidden, x0, target, params, velocity, grads,
                               params_bf16, lr, momentum, loss_out, workspace, eps=1e-6,
                               slope=0.5, stream=None):
    """mlp_stack_train_step with the kept block outputs in 8 bits."""
    _sizes(n_blocks, T, d, hidden)
    wsb = workspace.numel() * workspace.element_size()
    _check(load().mlp_stack_train_step_ckpt8(n_blocks, T, d, hidden, eps, slope, _ptr(x0),
                                             _ptr(target), _ptr(params), _ptr(velocity),
                                             _ptr(grads), _ptr(params_bf16), lr, momentum,
                                             _ptr(loss_out), _ptr(workspace), wsb,
                                             _stream(stream)), "mlp_stack_train_step_ckpt8")


# ------------------------------------------------------------------ feed-forward operators
#
# Matrices are 2-D CUDA tensors on the current device with unit stride along a
# row; their row pitch is taken from stride(0), so column slices of wider
# tensors are fine where the first column starts on 16 bytes (as every pointer
# has to).  Outputs are given by the caller.  `ckpt` is an 8-bit
# checkpoint: a pair (q, scale) of an int8 [rows, cols] and a uint8
# [rows, mlp_ckpt8_scale_cols(cols)] matrix.

# These checks run on every call, and a call of a few microseconds is mostly
# host time (layer norm of one row: 6.6 us, of which the launch is 3.2): they
# look at each property once, and take the stream's handle without making a
# Stream object (2.9 us).

_torch = None
_raw_stream = None
_FLOAT_CODES = {}


def _load_torch():
    global _torch, _raw_stream
    import torch
    # the current stream's handle without a Stream object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _FLOAT_CODES.update({torch.float32: MLP_DTYPE_F32, torch.bfloat16: MLP_DTYPE_BF16,
                         torch.float16: MLP_DTYPE_F16})
    _torch = torch


def _device(t, what):
    """The CUDA device of t, which must be the current one (launches and streams go there)."""
    if _torch is None:
        _load_torch()
    dev = t.get_device()
    if dev < 0 or dev != _torch.cuda.current_device():
        raise ValueError("%s must be on the current CUDA device (got %s)" % (what, t.device))
    return dev


# The C entry points take sizes and pitches as 32-bit ints, and ctypes would
# pass a larger one on by its low 32 bits.
_INT_MAX = 0x7fffffff


def _sizes(*n):
    """The sizes as they are, if each fits a 32-bit int."""
    if max(n) > _INT_MAX or min(n) < -_INT_MAX:
        raise ValueError("sizes and row pitches must be at most %d (got %s)" % (_INT_MAX, n))
    return n


def _mat(t, what, rows, cols, dev, dtype=None):
    """(address, row pitch) of a [rows, cols] matrix on device dev; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols):
        raise ValueError("%s must be [%d, %d] (got %s)" % (what, rows, cols, tuple(t.shape)))
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (what, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device (got %s)" % (what, t.device))
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s: the values of a row must be adjacent (strides %s)"
                         % (what, (pitch, step)))
    if rows <= 1:
        # the pitch of a single row is never used; a whole number of 16-byte
        # pieces keeps it acceptable for any width
        pitch = (cols + 15) // 16 * 16
    if (rows | cols | pitch) > _INT_MAX:  # none is negative
        _sizes(rows, cols, pitch)
    return t.data_ptr(), pitch


def _vec(t, what, n, dev):
    """Address of a contiguous fp32 vector of n values on device dev; None for None."""
    if t is None:
        return None
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be %d contiguous values (got %s)" % (what, n, tuple(t.shape)))
    if t.dtype is not _torch.float32:
        raise TypeError("%s must be torch.float32 (got %s)" % (what, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device (got %s)" % (what, t.device))
    return t.data_ptr()


def _ckpt(ckpt, what, rows, cols, dev):
    """(q address, pitch, scale address, pitch) of an 8-bit checkpoint."""
    if ckpt is None:
        return None, 0, None, 0
    q, scale = ckpt
    groups = (cols + MLP_CKPT8_GROUP - 1) // MLP_CKPT8_GROUP
    return (*_mat(q, what + " values", rows, cols, dev, _torch.int8),
            *_mat(scale, what + " scales", rows, groups, dev, _torch.uint8))


def _ws(t, dev):
    if t is None:
        return None, 0
    if t.get_device() != dev:
        raise ValueError("workspace must be on the current CUDA device (got %s)" % t.device)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _code_of(dtype):
    """MLP_DTYPE_* of a floating torch dtype."""
    if _torch is None:
        _load_torch()
    code = _FLOAT_CODES.get(dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % dtype)
    return code


def _stream_of(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def mlp_ckpt8_scale_cols(cols: int) -> int:
    """Scale bytes per row of an 8-bit checkpoint of `cols` columns."""
    return load().mlp_ckpt8_scale_cols(*_sizes(cols))


def mlp_ckpt8_encode(x, q, scale, stream=None):
    """x [rows, cols] (fp32, bf16 or fp16) into the 8-bit checkpoint (q, scale)."""
    T, d = x.shape
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", T, d, dev)
    qp, ldq, sp, lds = _ckpt((q, scale), "checkpoint", T, d, dev)
    _check(load().mlp_ckpt8_encode(xp, _code_of(x.dtype), T, d, ldx, qp, ldq, sp, lds,
                                   _stream_of(stream, dev)), "mlp_ckpt8_encode")


def mlp_ckpt8_decode(q, scale, out, stream=None):
    """The values of the 8-bit checkpoint (q, scale) into out (fp32, bf16 or fp16)."""
    T, d = out.shape
    dev = _device(out, "out")
    op, ldo = _mat(out, "out", T, d, dev)
    qp, ldq, sp, lds = _ckpt((q, scale), "checkpoint", T, d, dev)
    _check(load().mlp_ckpt8_decode(qp, ldq, sp, lds, T, d, op, _code_of(out.dtype), ldo,
                                   _stream_of(stream, dev)), "mlp_ckpt8_decode")


def mlp_layernorm_fwd(x, y, gain=None, shift=None, mean=None, rstd=None, ckpt=None, eps=1e-5,
                      stream=None):
    """Layer norm of the rows of x into y (same dtype); mean, rstd: fp32 [T]
    kept for the backward; ckpt: receives x in 8 bits."""
    T, d = x.shape
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", T, d, dev)
    yp, ldy = _mat(y, "y", T, d, dev, x.dtype)
    qp, ldq, sp, lds = _ckpt(ckpt, "ckpt", T, d, dev)
    _check(load().mlp_layernorm_fwd(xp, _code_of(x.dtype), ldx, _vec(gain, "gain", d, dev),
                                    _vec(shift, "shift", d, dev), T, d, eps, yp, ldy,
                                    _vec(mean, "mean", T, dev), _vec(rstd, "rstd", T, dev), qp,
                                    ldq, sp, lds, _stream_of(stream, dev)), "mlp_layernorm_fwd")


def mlp_layernorm_workspace_bytes(T: int, d: int) -> int:
    return load().mlp_layernorm_workspace_bytes(*_sizes(T, d))


def mlp_layernorm_bwd(dy, mean, rstd, dx, dgain, dshift, workspace, x=None, ckpt=None, gain=None,
                      dres=None, stream=None):
    """Backward of mlp_layernorm_fwd from its input x or the 8-bit checkpoint
    of it; dx (+ dres, the gradient past the norm), dgain and dshift fp32."""
    T, d = dy.shape
    dev = _device(dy, "dy")
    dyp, lddy = _mat(dy, "dy", T, d, dev)
    xp, ldx = _mat(x, "x", T, d, dev, dy.dtype)
    qp, ldq, sp, lds = _ckpt(ckpt, "ckpt", T, d, dev)
    rp, ldr = _mat(dres, "dres", T, d, dev, dy.dtype)
    dxp, lddx = _mat(dx, "dx", T, d, dev, dy.dtype)
    wp, wsb = _ws(workspace, dev)
    _check(load().mlp_layernorm_bwd(dyp, _code_of(dy.dtype), lddy, xp, ldx, qp, ldq, sp, lds,
                                    _vec(mean, "mean", T, dev), _vec(rstd, "rstd", T, dev),
                                    _vec(gain, "gain", d, dev), rp, ldr, T, d, dxp, lddx,
                                    _vec(dgain, "dgain", d, dev), _vec(dshift, "dshift", d, dev), wp,
                                    wsb, _stream_of(stream, dev)), "mlp_layernorm_bwd")


def mlp_linear_workspace_bytes(T: int, d_in: int, d_out: int, dtype) -> int:
    """Workspace of mlp_linear_fwd (0 for most shapes; fewer rows may need more);
    dtype: the operands' torch dtype."""
    return load().mlp_linear_workspace_bytes(*_sizes(T, d_in, d_out), _code_of(dtype))


def mlp_linear_fwd(x, w, y, bias=None, act=MLP_ACT_NONE, slope=0.5, residual=None, u=None,
                   ckpt=None, workspace=None, stream=None):
    """y = f(x w + bias) + residual; x [T, d_in], w [d_in, d_out]; y (and
    residual) of x's dtype or fp32; u: receives the pre-activations, ckpt:
    receives them in 8 bits."""
    T, k = x.shape
    n = w.shape[1]
    dev = _device(x, "x")
    xp, ldx = _mat(x, "x", T, k, dev)
    wp, ldw = _mat(w, "w", k, n, dev, x.dtype)
    yp, ldy = _mat(y, "y", T, n, dev)
    rp, ldr = _mat(residual, "residual", T, n, dev, y.dtype)
    up, ldu = _mat(u, "u", T, n, dev, x.dtype)
    qp, ldq, sp, lds = _ckpt(ckpt, "ckpt", T, n, dev)
    ws, wsb = _ws(workspace, dev)
    _check(load().mlp_linear_fwd(xp, ldx, wp, ldw, T, k, n, _code_of(x.dtype), _vec(bias, "bias", n, dev),
                                 act, slope, rp, ldr, yp, ldy, _code_of(y.dtype), up, ldu, qp, ldq,
                                 sp, lds, ws, wsb, _stream_of(stream, dev)), "mlp_linear_fwd")


def mlp_linear_bwd_workspace_bytes(T: int, d_in: int, d_out: int, dtype) -> int:
    """Workspace of mlp_linear_bwd for w [d_in, d_out] and dy [T, d_out] (fewer
    rows may need more)."""
    return load().mlp_linear_bwd_workspace_bytes(*_sizes(T, d_in, d_out), _code_of(dtype))


def mlp_linear_bwd(dy, w, du, act=MLP_ACT_NONE, slope=0.5, u=None, ckpt=None, dbias=None, a=None,
                   workspace=None, stream=None):
    """du = (dy w^T) f'(u); dy [T, d_out], w [d_in, d_out], u [T, d_in] given
    as it is or as an 8-bit checkpoint; dbias fp32 [d_in] receives the column
    sums of du, a (dy's dtype) the activations f(u)."""
    T, k = dy.shape
    n = w.shape[0]
    dev = _device(dy, "dy")
    dyp, lddy = _mat(dy, "dy", T, k, dev)
    wp, ldw = _mat(w, "w", n, k, dev, dy.dtype)
    dup, lddu = _mat(du, "du", T, n, dev)
    up, ldu = _mat(u, "u", T, n, dev, dy.dtype)
    qp, ldq, sp, lds = _ckpt(ckpt, "ckpt", T, n, dev)
    ap, lda = _mat(a, "a", T, n, dev, dy.dtype)
    ws, wsb = _ws(workspace, dev)
    _check(load().mlp_linear_bwd(dyp, lddy, wp, ldw, T, n, k, _code_of(dy.dtype), act, slope, up, ldu,
                                 qp, ldq, sp, lds, dup, lddu, _code_of(du.dtype),
                                 _vec(dbias, "dbias", n, dev), ap, lda, ws, wsb, _stream_of(stream, dev)),
           "mlp_linear_bwd")


def mlp_act_bwd_workspace_bytes(T: int, n: int) -> int:
    """Workspace of mlp_act_bwd with dbias (fewer rows may need more)."""
    return load().mlp_act_bwd_workspace_bytes(*_sizes(T, n))


def mlp_act_bwd(dy, du, act=MLP_ACT_NONE, slope=0.5, u=None, ckpt=None, dbias=None, a=None,
                workspace=None, stream=None):
    """du = dy f'(u) with the column sums and activations of mlp_linear_bwd,
    without a product (a layer whose own output has the activation)."""
    T, n = dy.shape
    dev = _device(dy, "dy")
    dyp, lddy = _mat(dy, "dy", T, n, dev)
    dup, lddu = _mat(du, "du", T, n, dev, dy.dtype)
    up, ldu = _mat(u, "u", T, n, dev, dy.dtype)
    qp, ldq, sp, lds = _ckpt(ckpt, "ckpt", T, n, dev)
    ap, lda = _mat(a, "a", T, n, dev, dy.dtype)
    ws, wsb = _ws(workspace, dev)
    _check(load().mlp_act_bwd(dyp, lddy, T, n, _code_of(dy.dtype), act, slope, up, ldu, qp, ldq, sp,
                              lds, dup, lddu, _vec(dbias, "dbias", n, dev), ap, lda, ws, wsb,
                              _stream_of(stream, dev)), "mlp_act_bwd")
