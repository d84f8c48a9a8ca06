"""ctypes binding of ``libvswin.so`` (``include/vswin.h``): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; PyTorch only owns
device memory and streams. There is no fallback: if the library is missing
or a call fails, a ``VswinError`` is raised.
"""

from __future__ import annotations

import array
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# VSWIN_LIBRARY may name another build of the same library (the in-tree
# libvswin_debug.so, built with VSWIN_DEBUG_BOUNDS) to load instead.
LIB_PATH = os.environ.get("VSWIN_LIBRARY") or os.path.join(_PKG, "libvswin.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NO_MEMORY, ERR_BOUNDS = range(7)
INJECT_CUDA, INJECT_ALLOC = 1, 2

# Every symbol include/vswin.h declares.
EXPORTS = (
    "vswin_wmsa_forward",
    "vswin_wmsa_forward_f32",
    "vswin_wmsa_forward_host",
    "vswin_wmsa_index_maps",
    "vswin_clamp_window",
    "vswin_last_error",
    "vswin_poll_error",
    "vswin_launch_count",
    "vswin_set_wait_limit_ns",
    "vswin_selftest_timeout",
    "vswin_version",
    "vswin_profile_enable",
    "vswin_profile_collect",
    "vswin_wmsa_forward_noalloc",
    "vswin_set_exact_softmax",
    "vswin_block_msa_forward",
    "vswin_wmsa_backward_f32",
    "vswin_wmsa_backward",
    "vswin_mlp_forward",
    "vswin_block_forward",
    "vswin_patch_merge_forward",
    "vswin_test_inject_failure",
    "vswin_debug_plant_row",
    "vswin_debug_bounds_enabled",
    "vswin_qk_norm_forward",
    "vswin_qk_norm_backward",
    "vswin_bucket_map",
    "vswin_bias_attention_forward",
    "vswin_bias_attention_backward",
    "vswin_adamw_step",
    "vswin_adamw_decode",
)

KERNEL_KINDS = ("qkv_gemm", "attention", "proj_gemm", "other", "mlp", "attention_bwd")


class VswinError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"vswin status {status}: {message}")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_IP = ctypes.POINTER(ctypes.c_int)
_LL = ctypes.c_longlong

# vswin_dtype
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
DTYPE_OF = {number: dtype for dtype, number in DTYPES.items()}
MAX_DISTANCE = 1 << 20  # of a bucket map
_INT_MAX = 2**31 - 1
ADAMW_BLOCK = 256  # elements that share one scale of the 8-bit moments


class _Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("batch_stride", _LL), ("token_stride", _LL), ("head_stride", _LL)]


class _Rotation(ctypes.Structure):
    _fields_ = [("cos", _P), ("sin", _P), ("rows", _I), ("dim", _I), ("interleaved", _I), ("positions", _P)]


class _BucketBias(ctypes.Structure):
    _fields_ = [("table", _P), ("map", _P), ("buckets", _I), ("max_distance", _I)]


class _Visibility(ctypes.Structure):
    _fields_ = [("q_lens", _P), ("kv_lens", _P), ("q_start", _P), ("causal", _I)]


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", _P), ("master", _P), ("grad", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("n", _LL), ("weight_decay", ctypes.c_double), ("param_dtype", _I), ("grad_dtype", _I)]


_data_ptr, _get_device, _is_contiguous = torch.Tensor.data_ptr, torch.Tensor.get_device, torch.Tensor.is_contiguous
_RECORD_WORDS, _GRAD_WORD = ctypes.sizeof(_AdamwTensor) // 8, _AdamwTensor.grad.offset // 8


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise VswinError(-1, f"{LIB_PATH} is missing: build it with "
                                 "`python -m shifted_window_attention_sw_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        layer = [_P, _I, _I, _I, _I, _I, _I, _IP, _IP, _P, _P, _P, _P, _P, _P, _P]
        for name in ("vswin_wmsa_forward", "vswin_wmsa_forward_f32", "vswin_wmsa_forward_host",
                     "vswin_wmsa_forward_noalloc"):
            fn = getattr(L, name)
            fn.argtypes = layer
            fn.restype = _I
        L.vswin_block_msa_forward.argtypes = layer[:9] + [_P, _P, ctypes.c_float] + layer[9:]
        L.vswin_block_msa_forward.restype = _I
        L.vswin_wmsa_backward_f32.argtypes = layer[:15] + [_P] * 6 + [_P]  # ..., dy, six gradients, stream
        L.vswin_wmsa_backward_f32.restype = _I
        L.vswin_wmsa_backward.argtypes = layer[:15] + [_P] * 6 + [_P]
        L.vswin_wmsa_backward.restype = _I
        L.vswin_mlp_forward.argtypes = [_P, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                                        _P]
        L.vswin_mlp_forward.restype = _I
        L.vswin_block_forward.argtypes = (layer[:9] + [_P, _P] + [_P] * 5 + [_P, _P, _I] + [_P] * 4 +
                                          [ctypes.c_float, _P, _P])
        L.vswin_block_forward.restype = _I
        L.vswin_patch_merge_forward.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, ctypes.c_float, _P, _P, _P, _P]
        L.vswin_patch_merge_forward.restype = _I
        L.vswin_wmsa_index_maps.argtypes = [_I, _I, _I, _I, _IP, _IP, _P, _P, _P, _P]
        L.vswin_wmsa_index_maps.restype = _I
        L.vswin_clamp_window.argtypes = [_I, _I, _I, _IP, _IP, _IP, _IP]
        L.vswin_clamp_window.restype = _I
        L.vswin_last_error.argtypes = []
        L.vswin_last_error.restype = ctypes.c_char_p
        L.vswin_poll_error.argtypes = [_P]
        L.vswin_poll_error.restype = _I
        L.vswin_launch_count.argtypes = []
        L.vswin_launch_count.restype = ctypes.c_ulonglong
        L.vswin_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.vswin_set_wait_limit_ns.restype = None
        L.vswin_set_exact_softmax.argtypes = [_I]
        L.vswin_set_exact_softmax.restype = None
        L.vswin_selftest_timeout.argtypes = [_P]
        L.vswin_selftest_timeout.restype = _I
        L.vswin_profile_enable.argtypes = [_I]
        L.vswin_profile_enable.restype = _I
        L.vswin_profile_collect.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_ulonglong), _I]
        L.vswin_profile_collect.restype = _I
        L.vswin_version.argtypes = []
        L.vswin_version.restype = _I
        L.vswin_test_inject_failure.argtypes = [_I, _I]
        L.vswin_test_inject_failure.restype = _I
        L.vswin_debug_plant_row.argtypes = [ctypes.c_longlong, _I]
        L.vswin_debug_plant_row.restype = _I
        L.vswin_debug_bounds_enabled.argtypes = []
        L.vswin_debug_bounds_enabled.restype = _I
        H, D = ctypes.POINTER(_Heads), ctypes.c_double
        norm = [_I] * 6 + [H, H, _P, _P, ctypes.c_float, ctypes.POINTER(_Rotation)]
        attn = [_I] * 7 + [H, H, H, ctypes.c_float, ctypes.POINTER(_BucketBias), ctypes.POINTER(_Visibility)]
        L.vswin_qk_norm_forward.argtypes = norm + [H, H, _P]
        L.vswin_qk_norm_backward.argtypes = norm + [H, H, H, H, _P, _P, _P]
        L.vswin_bucket_map.argtypes = [_I, _I, _I, _IP]
        L.vswin_bias_attention_forward.argtypes = attn + [H, _P, _P]
        L.vswin_bias_attention_backward.argtypes = attn + [H, _P, H, H, H, H, _P, _P]
        L.vswin_adamw_step.argtypes = [ctypes.POINTER(_AdamwTensor), _I, _I, D, D, D, D, _LL, _P, _P, _P]
        L.vswin_adamw_decode.argtypes = [_P, _P, _P, _P, _LL, _I, _P, _P, _P]
        for name in ("vswin_qk_norm_forward", "vswin_qk_norm_backward", "vswin_bucket_map",
                     "vswin_bias_attention_forward", "vswin_bias_attention_backward", "vswin_adamw_step",
                     "vswin_adamw_decode"):
            getattr(L, name).restype = _I
        _lib = L
    return _lib


def last_error() -> str:
    return lib().vswin_last_error().decode()


def _check(status):
    if status != OK:
        raise VswinError(status, last_error())


def _i3(v):
    v = tuple(int(a) for a in v)
    if len(v) != 3:
        raise ValueError("window and shift need 3 entries")
    return (ctypes.c_int * 3)(*v)


def _stream_handle(stream, device=None):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _layer_call(fn, x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out, stream, device=None):
    # the library launches on the current device, so make the tensors' device current
    B, T, H, W, C = x.shape
    dev = device or x.device
    with torch.cuda.device(dev):
        _check(fn(_ptr(x), B, T, H, W, C, int(heads), _i3(window), _i3(shift), _ptr(Wqkv), _ptr(bqkv),
                  _ptr(Wproj), _ptr(bproj), _ptr(table), _ptr(out), _stream_handle(stream, dev)))
    return out


def _prep(x, tensors, dtype, device=None):
    """dtype and contiguity of every tensor; with ``device``, that every tensor is a
    CUDA tensor on that device. The library reads raw pointers, so a host tensor or
    one on another GPU must be refused here."""
    for name, t in tensors.items():
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if device is not None:
        for name, t in tensors.items():
            if not t.is_cuda or t.device != device:
                raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")


def _table_rows(window):
    w = tuple(int(a) for a in window)
    if len(w) != 3:
        raise ValueError("window and shift need 3 entries")
    return (2 * w[0] - 1) * (2 * w[1] - 1) * (2 * w[2] - 1)


def _check_shapes(x, window, heads, Wqkv=None, bqkv=None, Wproj=None, bproj=None, table=None, **same_as_x):
    """Shapes the header fixes for a layer on x (B, T, H, W, C): Wqkv [C][3C], bqkv [3C],
    Wproj [C][C], bproj [C], bias_table [(2P-1)(2Mh-1)(2Mw-1)][heads]; every tensor in
    ``same_as_x`` has x's shape. The library trusts these sizes, so a short buffer would
    be read or written past its end."""
    if x.dim() != 5:
        raise ValueError(f"x must be (B, T, H, W, C), got shape {tuple(x.shape)}")
    C = x.shape[-1]
    want = {"Wqkv": (Wqkv, (C, 3 * C)), "bqkv": (bqkv, (3 * C,)), "Wproj": (Wproj, (C, C)),
            "bproj": (bproj, (C,)), "bias_table": (table, (_table_rows(window), int(heads)))}
    for name, (t, shape) in want.items():
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    for name, t in same_as_x.items():
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} must have the shape of x {tuple(x.shape)}, got {tuple(t.shape)}")


def _layer_args(x, window, heads, dtype, Wqkv, bqkv, Wproj, bproj, table, out, **more):
    tensors = dict(x=x, Wqkv=Wqkv, bqkv=bqkv, Wproj=Wproj, bproj=bproj, table=table, out=out, **more)
    _prep(x, tensors, dtype, x.device)
    _check_shapes(x, window, heads, Wqkv, bqkv, Wproj, bproj, table, out=out)


def wmsa_forward(x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out=None, stream=None):
    """bf16 layer forward on the GPU (tcgen05 path). All tensors bf16 on one CUDA device."""
    if out is None:
        out = torch.empty_like(x)
    _layer_args(x, window, heads, torch.bfloat16, Wqkv, bqkv, Wproj, bproj, table, out)
    return _layer_call(lib().vswin_wmsa_forward, x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out,
                       stream)


def block_msa_forward(x, window, shift, gamma, beta, eps, Wqkv, bqkv, Wproj, bproj, table, heads, out=None,
                      stream=None):
    """bf16 forward of a block's attention half, out = x + layer(LN(x)), with the
    norm and the residual fused into the layer's kernels. ``out`` may be ``x``."""
    if out is None:
        out = torch.empty_like(x)
    _layer_args(x, window, heads, torch.bfloat16, Wqkv, bqkv, Wproj, bproj, table, out, gamma=gamma, beta=beta)
    B, T, H, W, C = x.shape
    for name, t in (("gamma", gamma), ("beta", beta)):
        if tuple(t.shape) != (C,):
            raise ValueError(f"{name} must have shape ({C},), got {tuple(t.shape)}")
    with torch.cuda.device(x.device):
        _check(lib().vswin_block_msa_forward(
            _ptr(x), B, T, H, W, C, int(heads), _i3(window), _i3(shift), _ptr(gamma), _ptr(beta), float(eps),
            _ptr(Wqkv), _ptr(bqkv), _ptr(Wproj), _ptr(bproj), _ptr(table), _ptr(out),
            _stream_handle(stream, x.device)))
    return out


def mlp_forward(x, gamma, beta, eps, W1, b1, W2, b2, out=None, stream=None):
    """bf16 forward of a block's MLP half, out = x + GELU(LN(x) W1 + b1) W2 + b2, as one
    fused kernel. W1 [C][hidden], W2 [hidden][C]. ``out`` may be ``x``."""
    if out is None:
        out = torch.empty_like(x)
    _prep(x, dict(x=x, gamma=gamma, beta=beta, W1=W1, b1=b1, W2=W2, b2=b2, out=out), torch.bfloat16, x.device)
    if x.dim() != 5:
        raise ValueError(f"x must be (B, T, H, W, C), got shape {tuple(x.shape)}")
    B, T, H, W, C = x.shape
    if W1.dim() != 2 or W1.shape[0] != C:
        raise ValueError(f"W1 must have shape ({C}, hidden), got {tuple(W1.shape)}")
    hidden = W1.shape[1]
    want = {"gamma": (gamma, (C,)), "beta": (beta, (C,)), "b1": (b1, (hidden,)), "W2": (W2, (hidden, C)),
            "b2": (b2, (C,)), "out": (out, tuple(x.shape))}
    for name, (t, shape) in want.items():
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    with torch.cuda.device(x.device):
        _check(lib().vswin_mlp_forward(_ptr(x), B, T, H, W, C, int(hidden), _ptr(gamma), _ptr(beta), float(eps),
                                       _ptr(W1), _ptr(b1), _ptr(W2), _ptr(b2), _ptr(out),
                                       _stream_handle(stream, x.device)))
    return out


def block_forward(x, window, shift, attn, mlp, heads, eps=1e-5, out=None, stream=None):
    """bf16 forward of a whole block: z = x + layer(LN1(x)), out = z + MLP(LN2(z)).
    ``attn`` = dict(gamma, beta, Wqkv, bqkv, Wproj, bproj, table); ``mlp`` = dict(gamma, beta,
    W1, b1, W2, b2). ``out`` may be ``x``."""
    if out is None:
        out = torch.empty_like(x)
    _layer_args(x, window, heads, torch.bfloat16, attn["Wqkv"], attn["bqkv"], attn["Wproj"], attn["bproj"],
                attn["table"], out, gamma1=attn["gamma"], beta1=attn["beta"], gamma2=mlp["gamma"], beta2=mlp["beta"],
                W1=mlp["W1"], b1=mlp["b1"], W2=mlp["W2"], b2=mlp["b2"])
    B, T, H, W, C = x.shape
    hidden = mlp["W1"].shape[1] if mlp["W1"].dim() == 2 else -1
    want = {"gamma1": (attn["gamma"], (C,)), "beta1": (attn["beta"], (C,)), "gamma2": (mlp["gamma"], (C,)),
            "beta2": (mlp["beta"], (C,)), "W1": (mlp["W1"], (C, hidden)), "b1": (mlp["b1"], (hidden,)),
            "W2": (mlp["W2"], (hidden, C)), "b2": (mlp["b2"], (C,))}
    for name, (t, shape) in want.items():
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    with torch.cuda.device(x.device):
        _check(lib().vswin_block_forward(
            _ptr(x), B, T, H, W, C, int(heads), _i3(window), _i3(shift), _ptr(attn["gamma"]), _ptr(attn["beta"]),
            _ptr(attn["Wqkv"]), _ptr(attn["bqkv"]), _ptr(attn["Wproj"]), _ptr(attn["bproj"]), _ptr(attn["table"]),
            _ptr(mlp["gamma"]), _ptr(mlp["beta"]), int(hidden), _ptr(mlp["W1"]), _ptr(mlp["b1"]), _ptr(mlp["W2"]),
            _ptr(mlp["b2"]), float(eps), _ptr(out), _stream_handle(stream, x.device)))
    return out


def patch_merge_forward(x, gamma, beta, eps, Wr, br=None, out=None, stream=None):
    """bf16 patch merging: LN over each 2x2 spatial neighbourhood's 4C values, then
    Wr [4C][2C] (+ br). x (B, T, H, W, C) -> (B, T, ceil(H/2), ceil(W/2), 2C)."""
    if x.dim() != 5:
        raise ValueError(f"x must be (B, T, H, W, C), got shape {tuple(x.shape)}")
    B, T, H, W, C = x.shape
    oshape = (B, T, (H + 1) // 2, (W + 1) // 2, 2 * C)
    if out is None:
        out = torch.empty(oshape, dtype=x.dtype, device=x.device)
    tensors = dict(x=x, gamma=gamma, beta=beta, Wr=Wr, out=out)
    if br is not None:
        tensors["br"] = br
    _prep(x, tensors, torch.bfloat16, x.device)
    want = {"gamma": (gamma, (4 * C,)), "beta": (beta, (4 * C,)), "Wr": (Wr, (4 * C, 2 * C)), "out": (out, oshape)}
    if br is not None:
        want["br"] = (br, (2 * C,))
    for name, (t, shape) in want.items():
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    with torch.cuda.device(x.device):
        _check(lib().vswin_patch_merge_forward(_ptr(x), B, T, H, W, C, _ptr(gamma), _ptr(beta), float(eps),
                                               _ptr(Wr), _ptr(br), _ptr(out), _stream_handle(stream, x.device)))
    return out


def wmsa_backward_f32(x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, dy, stream=None):
    """fp32 gradients (dx, dWqkv, dbqkv, dWproj, dbproj, dtable) of the layer for output
    gradient ``dy``. All tensors float32 on one CUDA device."""
    _prep(x, dict(x=x, Wqkv=Wqkv, bqkv=bqkv, Wproj=Wproj, bproj=bproj, table=table, dy=dy), torch.float32,
          x.device)
    _check_shapes(x, window, heads, Wqkv, bqkv, Wproj, bproj, table, dy=dy)
    outs = [torch.empty_like(t) for t in (x, Wqkv, bqkv, Wproj, bproj, table)]
    B, T, H, W, C = x.shape
    with torch.cuda.device(x.device):
        _check(lib().vswin_wmsa_backward_f32(
            _ptr(x), B, T, H, W, C, int(heads), _i3(window), _i3(shift), _ptr(Wqkv), _ptr(bqkv), _ptr(Wproj),
            _ptr(bproj), _ptr(table), _ptr(dy), *[_ptr(o) for o in outs], _stream_handle(stream, x.device)))
    return tuple(outs)


def wmsa_backward(x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, dy, stream=None):
    """bf16 backward on the tensor cores: gradients (dx bf16; dWqkv, dbqkv, dWproj, dbproj,
    dtable float32) of the layer for output gradient ``dy``. Inputs bfloat16 on one CUDA
    device, as for wmsa_forward."""
    _prep(x, dict(x=x, Wqkv=Wqkv, bqkv=bqkv, Wproj=Wproj, bproj=bproj, table=table, dy=dy), torch.bfloat16,
          x.device)
    _check_shapes(x, window, heads, Wqkv, bqkv, Wproj, bproj, table, dy=dy)
    dx = torch.empty_like(x)
    grads = [torch.empty(t.shape, dtype=torch.float32, device=x.device) for t in (Wqkv, bqkv, Wproj, bproj, table)]
    B, T, H, W, C = x.shape
    with torch.cuda.device(x.device):
        _check(lib().vswin_wmsa_backward(
            _ptr(x), B, T, H, W, C, int(heads), _i3(window), _i3(shift), _ptr(Wqkv), _ptr(bqkv), _ptr(Wproj),
            _ptr(bproj), _ptr(table), _ptr(dy), _ptr(dx), *[_ptr(t) for t in grads], _stream_handle(stream, x.device)))
    return (dx, *grads)


def wmsa_forward_noalloc(x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out=None, stream=None):
    """bf16 layer forward that allocates no device memory: the library's fixed
    32 MiB scratch array is used instead (see include/vswin.h). ``out`` should be
    passed in by callers that cannot allocate; if it is None a tensor is created."""
    if out is None:
        out = torch.empty_like(x)
    _layer_args(x, window, heads, torch.bfloat16, Wqkv, bqkv, Wproj, bproj, table, out)
    return _layer_call(lib().vswin_wmsa_forward_noalloc, x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads,
                       out, stream)


def wmsa_forward_f32(x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out=None, stream=None):
    """fp32 layer forward on the GPU (FP32 FMA path). All tensors float32 on one CUDA device."""
    if out is None:
        out = torch.empty_like(x)
    _layer_args(x, window, heads, torch.float32, Wqkv, bqkv, Wproj, bproj, table, out)
    return _layer_call(lib().vswin_wmsa_forward_f32, x, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads,
                       out, stream)


def wmsa_forward_host(x_host, window, shift, Wqkv, bqkv, Wproj, bproj, table, heads, out_host, stream=None):
    """bf16 forward with x and out in host memory (copies inside the call; synchronises)."""
    _prep(x_host, dict(x_host=x_host, out_host=out_host), torch.bfloat16)
    for name, t in (("x_host", x_host), ("out_host", out_host)):
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor")
    dev = Wqkv.device
    _prep(x_host, dict(Wqkv=Wqkv, bqkv=bqkv, Wproj=Wproj, bproj=bproj, table=table), torch.bfloat16, dev)
    _check_shapes(x_host, window, heads, Wqkv, bqkv, Wproj, bproj, table, out_host=out_host)
    return _layer_call(lib().vswin_wmsa_forward_host, x_host, window, shift, Wqkv, bqkv, Wproj, bproj, table,
                       heads, out_host, stream, dev)


# ------------------------------------------------------------------ token sequences
def _refuse(name, t, shape, dtype, device):
    """Say what is wrong with a tensor that is not of this shape and type on this CUDA device. ``name`` is a text,
    or a list's name and an index in it."""
    name = name if isinstance(name, str) else f"{name[0]}[{name[1]}]"
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous (its channels, if it has heads), got strides {t.stride()}")


def _heads(name, t, shape, dtype, device):
    """View of a (B, L, heads, d) tensor; its channels have to be contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(name, t, shape, dtype, device)
    strides = t.stride()
    if strides[3] != 1 and shape[3] > 1:
        _refuse(name, t, shape, dtype, device)
    return _Heads(t.data_ptr(), *strides[:3])


def _flat(name, t, shape, dtype, device):
    """Pointer of a contiguous tensor of a given shape and type, None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(name, t, shape, dtype, device)
    return t.data_ptr()


def _run(fn, dev, stream, *args):
    """Calls an entry on a device's stream (its current one by default), with that device current."""
    # (the raw forms of torch.cuda.current_stream and current_device: these calls take a few us in all)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != OK:
        raise VswinError(status, last_error())


def _new(stream, like, shape=None, dtype=None):
    """Contiguous memory for a result, of a tensor's shape and type or of others on its device, from the stream
    that the call runs on."""
    # (the cheapest of torch's ways: 1.4 us for a shape like the tensor's, 1.9 for another, 2.4 for torch.empty)
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(None, like, shape, dtype)
    if shape is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    return like.new_empty(shape, dtype=dtype)


def _qk_norm_args(q, k, gamma_q, gamma_k, eps, cos, sin, positions, interleaved):
    shape, k_shape = q.shape, k.shape
    if len(shape) != 4 or len(k_shape) != 4:
        raise ValueError(f"q and k must be (B, L, heads, d), got {tuple(shape)} and {tuple(k_shape)}")
    B, L, hq, d = shape
    hk, dt, dev = k_shape[2], q.dtype, q.device
    if max(*shape, hk) > _INT_MAX:  # (ctypes would pass the low 32 bits)
        raise VswinError(ERR_UNSUPPORTED, f"sizes of q {tuple(shape)} or k {tuple(k_shape)} exceed 2^31 - 1")
    code = DTYPES.get(dt)
    if code is None:
        raise TypeError(f"q must be one of {list(DTYPES)}, got {dt}")
    if not q.is_cuda:
        _refuse("q", q, shape, dt, dev)
    rot = None
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2:
            raise ValueError("cos and sin must both be (rows, dim / 2)")
        angles = tuple(cos.shape)
        rot = _Rotation(_flat("cos", cos, angles, torch.float32, dev), _flat("sin", sin, angles, torch.float32, dev),
                        angles[0], 2 * angles[1], 1 if interleaved else 0,
                        _flat("positions", positions, (B, L), torch.int32, dev))
    elif positions is not None:
        raise ValueError("positions need cos and sin")
    return (B, L, hq, hk, d, dt, dev), [code, B, L, hq, hk, d, _heads("q", q, shape, dt, dev),
                                        _heads("k", k, (B, L, hk, d), dt, dev),
                                        _flat("gamma_q", gamma_q, (d,), dt, dev),
                                        _flat("gamma_k", gamma_k, (d,), dt, dev), float(eps), rot]


def qk_norm_forward(q, k, gamma_q, gamma_k, eps=1e-6, cos=None, sin=None, positions=None, interleaved=False,
                    q_out=None, k_out=None, stream=None):
    """Norm of every head of q (B, L, hq, d) and k (B, L, hk, d) over its d channels, times gamma [d], then
    the rotation of the first 2 * cos.shape[1] channels by row ``positions[b, l]`` (int32; row l without
    them) of the float32 tables cos and sin, in one pass; bf16, fp16 or fp32. Views with contiguous channels
    are taken as they are. ``q_out`` may be ``q`` and ``k_out`` ``k``. Returns (q_out, k_out)."""
    (B, L, hq, hk, d, dt, dev), args = _qk_norm_args(q, k, gamma_q, gamma_k, eps, cos, sin, positions, interleaved)
    q_out = _new(stream, q) if q_out is None else q_out
    k_out = _new(stream, k) if k_out is None else k_out
    _run(lib().vswin_qk_norm_forward, dev, stream, *args, _heads("q_out", q_out, (B, L, hq, d), dt, dev),
         _heads("k_out", k_out, (B, L, hk, d), dt, dev))
    return q_out, k_out


def qk_norm_backward(q, k, gamma_q, gamma_k, dq_out, dk_out, eps=1e-6, cos=None, sin=None, positions=None,
                     interleaved=False, dq=None, dk=None, stream=None):
    """Gradients (dq, dk in the type of q; dgamma_q, dgamma_k float32) of qk_norm_forward for the output
    gradients ``dq_out`` and ``dk_out``. ``dq`` and ``dk`` may be given, e.g. as slices of one buffer."""
    (B, L, hq, hk, d, dt, dev), args = _qk_norm_args(q, k, gamma_q, gamma_k, eps, cos, sin, positions, interleaved)
    dq = _new(stream, q) if dq is None else dq
    dk = _new(stream, k) if dk is None else dk
    dgamma = _new(stream, q, (2, d), torch.float32)
    at = dgamma.data_ptr()
    _run(lib().vswin_qk_norm_backward, dev, stream, *args, _heads("dq_out", dq_out, (B, L, hq, d), dt, dev),
         _heads("dk_out", dk_out, (B, L, hk, d), dt, dev), _heads("dq", dq, (B, L, hq, d), dt, dev),
         _heads("dk", dk, (B, L, hk, d), dt, dev), at, at + 4 * d)
    return dq, dk, dgamma[0], dgamma[1]


def bucket_map(buckets, max_distance, bidirectional=True, device="cuda"):
    """int32 tensor [2 * max_distance + 1]: the bucket of each offset key - query in [-max_distance,
    max_distance] (see vswin_bucket_map), as the attention with bucketed bias takes it."""
    # (the library refuses what lies outside; ctypes would pass the low 32 bits of more)
    buckets, max_distance = min(max(int(buckets), 0), _INT_MAX), min(max(int(max_distance), 0), MAX_DISTANCE + 1)
    out = torch.empty(2 * max_distance + 1, dtype=torch.int32)
    _check(lib().vswin_bucket_map(buckets, max_distance, 1 if bidirectional else 0, ctypes.cast(out.data_ptr(), _IP)))
    return out.to(device)


def _bias_attention_args(q, k, v, table, bucket_map, scale, causal, q_lens, kv_lens, q_start):
    shape, k_shape, table_shape, map_shape = q.shape, k.shape, table.shape, bucket_map.shape
    if len(shape) != 4 or len(k_shape) != 4:
        raise ValueError(f"q and k must be (B, L, heads, d), got {tuple(shape)} and {tuple(k_shape)}")
    B, Lq, hq, d = shape
    Lk, hk, dt, dev = k_shape[1], k_shape[2], q.dtype, q.device
    if max(*shape, Lk, hk) > _INT_MAX:  # (ctypes would pass the low 32 bits)
        raise VswinError(ERR_UNSUPPORTED, f"sizes of q {tuple(shape)} or k {tuple(k_shape)} exceed 2^31 - 1")
    code = DTYPES.get(dt)
    if code is None:
        raise TypeError(f"q must be torch.bfloat16 or torch.float16, got {dt}")
    if not q.is_cuda:
        _refuse("q", q, shape, dt, dev)
    if len(table_shape) != 2 or len(map_shape) != 1 or map_shape[0] % 2 == 0:
        raise ValueError("table must be (buckets, heads of q) and bucket_map (2 * max_distance + 1,), got "
                         f"{tuple(table_shape)} and {tuple(map_shape)}")
    buckets, D, ks = table_shape[0], map_shape[0] // 2, (B, Lk, hk, d)
    views = (_heads("q", q, shape, dt, dev), _heads("k", k, ks, dt, dev), _heads("v", v, ks, dt, dev))
    bias = _BucketBias(_flat("table", table, (buckets, hq), dt, dev),
                       _flat("bucket_map", bucket_map, (2 * D + 1,), torch.int32, dev), buckets, D)
    vis = _Visibility(_flat("q_lens", q_lens, (B,), torch.int32, dev), _flat("kv_lens", kv_lens, (B,), torch.int32, dev),
                      _flat("q_start", q_start, (B,), torch.int32, dev), 1 if causal else 0)
    scale = d ** -0.5 if scale is None else float(scale)
    return (B, Lq, Lk, hq, hk, d, dt, dev), [code, B, Lq, Lk, hq, hk, d, *views, scale, bias, vis]


def bias_attention_forward(q, k, v, table, bucket_map, scale=None, causal=False, q_lens=None, kv_lens=None,
                           q_start=None, out=None, lse=None, stream=None):
    """Attention of q (B, Lq, hq, d) over k, v (B, Lk, hk, d) with the bias table[bucket_map[key - position]][head];
    bf16 or fp16, d 32, 64 or 128, hq a multiple of hk. Query i of sequence b stands at position q_start[b] + i;
    it sees the keys below kv_lens[b] (with ``causal`` up to its own position), rows from q_lens[b] on are zero
    (int32 tensors [B], default: all). ``scale`` defaults to d ** -0.5. One new token of each sequence against a
    cache: Lq = 1, q_start = kv_lens - 1. Returns (out, lse), lse float32 (B, hq, Lq)."""
    (B, Lq, Lk, hq, hk, d, dt, dev), args = _bias_attention_args(q, k, v, table, bucket_map, scale, causal, q_lens,
                                                                 kv_lens, q_start)
    out = _new(stream, q) if out is None else out
    lse = _new(stream, q, (B, hq, Lq), torch.float32) if lse is None else lse
    _run(lib().vswin_bias_attention_forward, dev, stream, *args, _heads("out", out, (B, Lq, hq, d), dt, dev),
         _flat("lse", lse, (B, hq, Lq), torch.float32, dev))
    return out, lse


def bias_attention_backward(q, k, v, table, bucket_map, out, lse, dout, scale=None, causal=False, q_lens=None,
                            kv_lens=None, q_start=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv, dtable, all in the type of q) of bias_attention_forward for the output gradient
    ``dout``, from its ``out`` and ``lse``. ``dq``, ``dk`` and ``dv`` may be given, e.g. as slices of one buffer.
    In fp16 a small ``dout`` has to be scaled up first (see vswin_bias_attention_backward)."""
    (B, Lq, Lk, hq, hk, d, dt, dev), args = _bias_attention_args(q, k, v, table, bucket_map, scale, causal, q_lens,
                                                                 kv_lens, q_start)
    qs, ks = (B, Lq, hq, d), (B, Lk, hk, d)
    dq, dk, dv = (_new(stream, like) if t is None else t for t, like in ((dq, q), (dk, k), (dv, v)))
    dtable = _new(stream, table)
    _run(lib().vswin_bias_attention_backward, dev, stream, *args, _heads("out", out, qs, dt, dev),
         _flat("lse", lse, (B, hq, Lq), torch.float32, dev), _heads("dout", dout, qs, dt, dev),
         _heads("dq", dq, qs, dt, dev), _heads("dk", dk, ks, dt, dev), _heads("dv", dv, ks, dt, dev), dtable.data_ptr())
    return dq, dk, dv, dtable


# ------------------------------------------------------------------ optimizer
class AdamW:
    """AdamW over a list of contiguous weights on one CUDA device (see vswin_adamw_step): every step is one
    launch per 192 tensors. The object owns the moments (zeros, or the ones given) and keeps the weights' list.
    A weight may get another storage (``p.data = ...``), and a moment, scale or master is loaded by copying into it
    or by putting another tensor of its shape and type in its list (``m``, ``v``, ``m_scale``, ``v_scale``, ``master``);
    a captured step keeps the storages that it was captured with.

    weight_decay: one value or one per weight. bits: 32 (float32 moments) or 8 (codes with a scale per 256
    elements). master: float32 copies that are stepped and rounded into the weights: True makes them, or a list.
    moments: (m, v) lists to go on from, with ``scales`` (m_scale, v_scale) for 8 bits."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, master=None,
                 moments=None, scales=None):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if bits not in (8, 32):
            raise ValueError(f"bits must be 32 or 8, got {bits}")
        self.lr, self.betas, self.eps, self.bits, self.steps = lr, tuple(betas), eps, bits, 0
        dev = self.device = self.params[0].device
        if not self.params[0].is_cuda:
            _refuse("params[0]", self.params[0], self.params[0].shape, self.params[0].dtype, dev)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(self.params)
        if len(decay) != len(self.params):
            raise ValueError(f"{len(decay)} weight decays for {len(self.params)} parameters")
        if moments is None and scales is not None:
            raise ValueError("scales need moments")
        if moments is not None and bits == 8 and scales is None:
            raise ValueError("8-bit moments need their scales")

        def state(given, which, dtype, shape_of):
            if given is not None:
                return self._list(f"{which}", given[0 if which.startswith("m") else 1])
            return [torch.zeros(shape_of(p), dtype=dtype, device=dev) for p in self.params]

        full = lambda p: tuple(p.shape)  # noqa: E731
        blocks = lambda p: (-(-p.numel() // ADAMW_BLOCK),)  # noqa: E731
        mt, vt = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
        self.m, self.v = state(moments, "m", mt, full), state(moments, "v", vt, full)
        scales = scales if bits == 8 else None
        self.m_scale = state(scales, "m_scale", torch.float32, blocks) if bits == 8 else None
        self.v_scale = state(scales, "v_scale", torch.float32, blocks) if bits == 8 else None
        if master is True:
            master = [p.detach().float() for p in self.params]
            master = [t.clone() if t.data_ptr() == p.data_ptr() else t for t, p in zip(master, self.params)]
        self.master = None if not master else self._list("master", master)
        # the library's records, whose 8-byte words a step fills a column at a time
        words = bytearray(len(self.params) * ctypes.sizeof(_AdamwTensor))
        self._records = (_AdamwTensor * len(self.params)).from_buffer(words)
        self._words = memoryview(words).cast("q")
        for i, (p, r) in enumerate(zip(self.params, self._records)):
            dt = DTYPES.get(p.dtype)
            if dt is None:
                raise TypeError(f"params[{i}] must be one of {list(DTYPES)}, got {p.dtype}")
            r.n, r.weight_decay, r.param_dtype = p.numel(), decay[i], dt
        self._shapes = [p.shape for p in self.params]
        self._indices = [dev.index] * len(self.params)
        self._grad_types = None
        self._record()

    def _lists(self):
        return self.params, self.m, self.v, self.m_scale, self.v_scale, self.master

    def _addresses(self):
        every = [*self.params, *self.m, *self.v]
        if self.m_scale:
            every += [*self.m_scale, *self.v_scale]
        if self.master:
            every += self.master
        return list(map(_data_ptr, every))

    def _record(self):
        """Fills the records from the lists of weights and states as they are now."""
        self._recorded, count = None, len(self._shapes)  # (until every record is right)
        states = (torch.float32, torch.float32) if self.bits == 32 else (torch.int8, torch.uint8)
        scales = [(-(-r.n // ADAMW_BLOCK),) for r in self._records] if self.bits == 8 else self._shapes
        weights = [DTYPE_OF[r.param_dtype] for r in self._records]
        held = []
        for name, tensors, shapes, types in zip(
                ("params", "m", "v", "m_scale", "v_scale", "master"), self._lists(),
                (self._shapes, self._shapes, self._shapes, scales, scales, self._shapes),
                (weights, *([t] * count for t in (*states, torch.float32, torch.float32, torch.float32)))):
            if tensors is None:
                at = [0] * count
            else:
                tensors = self._list(name, tensors)
                if ([t.shape for t in tensors] != shapes or [t.dtype for t in tensors] != types
                        or list(map(_get_device, tensors)) != self._indices or not all(map(_is_contiguous, tensors))):
                    for i, t in enumerate(tensors):
                        _flat((name, i), t, shapes[i], types[i], self.device)
                at = list(map(_data_ptr, tensors))
                held.append(tensors)
            field = _AdamwTensor.param if name == "params" else getattr(_AdamwTensor, name)
            self._words[field.offset // 8::_RECORD_WORDS] = array.array("q", at)
        if len({r.param for r in self._records if r.n}) < sum(1 for r in self._records if r.n):
            raise ValueError("a weight stands in params twice")
        # (held, so that another tensor in a list has another address)
        self._held, self._recorded = held, self._addresses()

    def _list(self, name, tensors):
        tensors = list(tensors)
        if len(tensors) != len(self.params):
            raise ValueError(f"{name}: {len(tensors)} tensors for {len(self.params)} parameters")
        return tensors

    def step(self, grads, lr=None, step=None, grad_scale=None, stream=None):
        """One step with ``grads`` (contiguous, shaped as the weights; bf16, fp16 or fp32). ``step`` counts from 1
        (default: one more than the last call's) or is a one-element int32 CUDA tensor, read when the step runs, as a
        captured step needs (its lr and decays are the capture's; replays do not count in ``steps``). grad_scale: one-element float32 CUDA tensor that multiplies every gradient."""
        grads = self._list("grads", grads)
        dev = self.device
        types = [g.dtype for g in grads]
        if ([g.shape for g in grads] != self._shapes or list(map(_get_device, grads)) != self._indices
                or not all(map(_is_contiguous, grads))
                or types != self._grad_types and not DTYPES.keys() >= set(types)):
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):
                if g.dtype not in DTYPES or g.shape != shape or g.device != dev or not g.is_contiguous():
                    raise ValueError(f"grads[{i}] must be a contiguous {tuple(shape)} tensor of {list(DTYPES)} on "
                                     f"{dev}, got {g.dtype} {tuple(g.shape)} on {g.device}")
        if types != self._grad_types:
            for r, dtype in zip(self._records, types):
                r.grad_dtype = DTYPES[dtype]
            self._grad_types = types
        self._words[_GRAD_WORD::_RECORD_WORDS] = array.array("q", list(map(_data_ptr, grads)))
        if self._addresses() != self._recorded:  # some weight's or state's storage was exchanged
            self._record()
        count, count_dev = self.steps + 1, None
        if step is None:
            pass
        elif type(step) is not int and isinstance(step, torch.Tensor):  # (the check of a tensor's class is a slow one)
            count_dev = _flat("step", step, tuple(step.shape), torch.int32, dev)
            if step.numel() != 1:
                raise ValueError("step must have one element")
        else:
            count = int(step)
        if grad_scale is not None and grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one element")
        gs = None if grad_scale is None else _flat("grad_scale", grad_scale, tuple(grad_scale.shape), torch.float32, dev)
        _run(lib().vswin_adamw_step, dev, stream, self._records, len(self._records), self.bits,
             self.lr if lr is None else lr, *self.betas, self.eps, count, count_dev, gs)
        self.steps = count
        return self

    def moments(self, dtype=torch.float32, stream=None):
        """(m, v) lists of the moments' values: the states themselves for 32 bits, decoded copies for 8."""
        if self.bits == 32:
            return self.m, self.v
        pairs = [adamw_decode(*t, dtype=dtype, stream=stream)
                 for t in zip(self.m, self.m_scale, self.v, self.v_scale)]
        return [a for a, _ in pairs], [b for _, b in pairs]


def adamw_decode(m, m_scale, v, v_scale, dtype=torch.float32, stream=None):
    """(m, v) that 8-bit moments stand for: codes int8 and uint8 of one shape, scales float32 per 256 elements."""
    dev, shape = m.device, tuple(m.shape)
    if not m.is_cuda:
        _refuse("m", m, m.shape, m.dtype, dev)
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be one of {list(DTYPES)}, got {dtype}")
    blocks = (-(-m.numel() // ADAMW_BLOCK),)
    args = (_flat("m", m, shape, torch.int8, dev), _flat("m_scale", m_scale, blocks, torch.float32, dev),
            _flat("v", v, shape, torch.uint8, dev), _flat("v_scale", v_scale, blocks, torch.float32, dev))
    mo, vo = _new(stream, m, shape, dtype), _new(stream, m, shape, dtype)
    _run(lib().vswin_adamw_decode, dev, stream, *args, m.numel(), DTYPES[dtype], mo.data_ptr(), vo.data_ptr())
    return mo, vo


def index_maps(B, T, H, W, window, shift, device="cuda", stream=None):
    """(win_src, region, bias_idx) as int32 device tensors."""
    nW = 1
    N = 1
    for L, w in zip((T, H, W), window):
        nW *= -(-L // w)
        N *= w
    win_src = torch.empty(B * nW * N, dtype=torch.int32, device=device)
    region = torch.empty(nW * N, dtype=torch.int32, device=device)
    bias_idx = torch.empty(N * N, dtype=torch.int32, device=device)
    dev = win_src.device
    if not win_src.is_cuda:
        raise ValueError(f"index maps are written on a CUDA device, got {dev}")
    with torch.cuda.device(dev):
        _check(lib().vswin_wmsa_index_maps(B, T, H, W, _i3(window), _i3(shift), _ptr(win_src), _ptr(region),
                                           _ptr(bias_idx), _stream_handle(stream, dev)))
    return win_src, region, bias_idx


def clamp_window(T, H, W, window, shift):
    wo = (ctypes.c_int * 3)()
    so = (ctypes.c_int * 3)()
    _check(lib().vswin_clamp_window(T, H, W, _i3(window), _i3(shift), wo, so))
    return tuple(wo), tuple(so)


def poll_error(stream=None) -> int:
    """Synchronise and return the device error status (0 = OK, 4 = a kernel wait gave up,
    6 = a length, position or bucket that an operator over sequences read was out of range, or
    an index check of a VSWIN_DEBUG_BOUNDS build failed)."""
    return int(lib().vswin_poll_error(_stream_handle(stream)))


def launch_count() -> int:
    return int(lib().vswin_launch_count())


def set_wait_limit_ns(ns: int) -> None:
    lib().vswin_set_wait_limit_ns(int(ns))


def set_exact_softmax(on: bool) -> None:
    """Test hook: route every query row of the bf16 (P,7,7) kernel through its exact softmax path."""
    lib().vswin_set_exact_softmax(1 if on else 0)


def selftest_timeout(stream=None) -> None:
    _check(lib().vswin_selftest_timeout(_stream_handle(stream)))


def profile_enable(on: bool) -> None:
    _check(lib().vswin_profile_enable(1 if on else 0))


def profile_collect():
    """{kind: (total ms, launches)} for the launches recorded since the last collect."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_ulonglong * n)()
    _check(lib().vswin_profile_collect(ms, cnt, n))
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def version() -> int:
    return int(lib().vswin_version())


def inject_failure(kind: int, count: int = 1) -> None:
    """Test hook: the next `count` entry calls fail as a CUDA call would (INJECT_CUDA) or
    the next `count` scratch allocations fail (INJECT_ALLOC); count 0 clears."""
    _check(lib().vswin_test_inject_failure(int(kind), int(count)))


def debug_bounds_enabled() -> bool:
    return bool(lib().vswin_debug_bounds_enabled())


def debug_plant_row(slot: int, token: int) -> None:
    """Test hook of VSWIN_DEBUG_BOUNDS builds: every following bf16 layer forward
    overwrites its row-table entry for layer slot `slot` with `token` (slot < 0: off)."""
    _check(lib().vswin_debug_plant_row(int(slot), int(token)))
