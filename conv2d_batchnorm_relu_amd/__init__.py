"""Fused Conv2D -> BatchNorm -> ReLU (CBR) for AMD Instinct MI355X (gfx950).

A thin ctypes binding over ``libcbr.so`` (the HIP kernels and the C ABI declared in
``include/cbr.h``).  The functions carry the C names and only marshal arguments: torch
tensors are passed by device pointer, the stream defaults to torch's current stream.
All computation runs in the library's kernels; there is no CPU path, and every call
raises if the library has not been built.

Tensor conventions (see include/cbr.h): NHWC activations and KRSC filters as
``torch.bfloat16`` (or 16-bit integer tensors holding bf16 bits), float32 per-channel
vectors, an int32/uint32 packed ReLU mask of ``cbr_mask_words(shape)`` words, and a
caller-allocated device workspace of ``cbr_workspace_bytes(shape, op)`` bytes.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["CbrError", "CbrShape", "make_shape", "cbr_status_str", "cbr_output_hw", "cbr_mask_words",
           "cbr_workspace_bytes", "cbr_forward_train", "cbr_forward_infer", "cbr_backward",
           "cbr_conv2d_bias_relu", "cbr_conv2d_bias", "cbr_forward_train_noalloc",
           "CBR_OP_TRAIN", "CBR_OP_INFER", "CBR_OP_BWD", "library_path",
           "CbrBlockShape", "make_block_shape", "cbr_block_norm_workspace_bytes", "cbr_block_norm_forward",
           "cbr_block_norm_backward", "CbrQuantShape", "make_quant_shape", "cbr_fp8_quantize", "CbrGemmShape",
           "make_gemm_shape", "cbr_gemm_fp8_workspace_bytes", "cbr_gemm_fp8", "CBR_BF16", "CBR_F16", "CBR_F32",
           "CBR_E4M3", "CBR_E5M2", "CBR_NORM_NONE", "CBR_NORM_RMS", "CBR_NORM_LAYER"]

CBR_OP_TRAIN, CBR_OP_INFER, CBR_OP_BWD = 0, 1, 2
CBR_BF16, CBR_F16, CBR_F32, CBR_E4M3, CBR_E5M2 = 0, 1, 2, 3, 4
CBR_NORM_NONE, CBR_NORM_RMS, CBR_NORM_LAYER = 0, 1, 2
_BYTES = {CBR_BF16: 2, CBR_F16: 2, CBR_F32: 4, CBR_E4M3: 1, CBR_E5M2: 1}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libcbr.so")


class CbrShape(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in
                ("n", "h", "w", "c", "k", "r", "s", "stride_h", "stride_w", "pad_h", "pad_w")]


class CbrBlockShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("rows_per_gate", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("post", ctypes.c_int32), ("pre", ctypes.c_int32), ("stream_type", ctypes.c_int32),
                ("branch_type", ctypes.c_int32), ("alpha", ctypes.c_float), ("eps_post", ctypes.c_float),
                ("eps_pre", ctypes.c_float)]


class CbrQuantShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ldq", ctypes.c_int64),
                ("src_type", ctypes.c_int32), ("q_type", ctypes.c_int32), ("transpose", ctypes.c_int32),
                ("block", ctypes.c_int32)]


class CbrGemmShape(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("lda", ctypes.c_int64),
                ("ldb", ctypes.c_int64), ("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32),
                ("d_type", ctypes.c_int32), ("b_block", ctypes.c_int32), ("relu", ctypes.c_int32),
                ("short_sums", ctypes.c_int32)]


class CbrError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str | None = None):
        self.status = status
        msg = detail if detail is not None else cbr_status_str(status)
        super().__init__(f"{where}: {msg} (status {status})")


_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(the CBR operator has no CPU fallback)")
    # The library must resolve its HIP runtime to the one that owns the callers' device
    # memory and streams.  torch loads its own copy of the runtime; loading torch first
    # makes the library bind to that copy (same soname) instead of a second one.
    import torch  # noqa: F401
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    S = ctypes.POINTER(CbrShape)
    lib.cbr_status_str.argtypes = [ctypes.c_int]
    lib.cbr_status_str.restype = ctypes.c_char_p
    lib.cbr_output_hw.argtypes = [S, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.cbr_output_hw.restype = ctypes.c_int
    lib.cbr_mask_words.argtypes = [S]
    lib.cbr_mask_words.restype = ctypes.c_size_t
    lib.cbr_workspace_bytes.argtypes = [S, ctypes.c_int]
    lib.cbr_workspace_bytes.restype = ctypes.c_size_t
    lib.cbr_forward_train.argtypes = [S, P, P, P, P, P, P, ctypes.c_float, ctypes.c_float,
                                      P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.cbr_forward_train.restype = ctypes.c_int
    lib.cbr_forward_infer.argtypes = [S, P, P, P, P, P, P, P, ctypes.c_float, P, P, ctypes.c_size_t, P]
    lib.cbr_forward_infer.restype = ctypes.c_int
    lib.cbr_backward.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.cbr_backward.restype = ctypes.c_int
    lib.cbr_forward_train_ev.argtypes = lib.cbr_forward_train.argtypes + [P]
    lib.cbr_forward_train_ev.restype = ctypes.c_int
    lib.cbr_forward_infer_ev.argtypes = lib.cbr_forward_infer.argtypes + [P]
    lib.cbr_forward_infer_ev.restype = ctypes.c_int
    lib.cbr_backward_ev.argtypes = lib.cbr_backward.argtypes + [P]
    lib.cbr_backward_ev.restype = ctypes.c_int
    lib.cbr_forward_train_noalloc.argtypes = [S, P, P, P, P, P, P, ctypes.c_float, ctypes.c_float,
                                              P, P, P, P, P, P, P, P]
    lib.cbr_forward_train_noalloc.restype = ctypes.c_int
    for name in ("cbr_conv2d_bias_relu", "cbr_conv2d_bias"):
        fn, fe = getattr(lib, name), getattr(lib, name + "_ev")
        fn.argtypes = [S, P, P, P, P, P]
        fn.restype = ctypes.c_int
        fe.argtypes = fn.argtypes + [P]
        fe.restype = ctypes.c_int
    B, U, G = (ctypes.POINTER(t) for t in (CbrBlockShape, CbrQuantShape, CbrGemmShape))
    for name, args, res in (
            ("cbr_block_norm_workspace_bytes", [B], ctypes.c_size_t),
            ("cbr_block_norm_forward", [B] + [P] * 13, ctypes.c_int),
            ("cbr_block_norm_backward", [B] + [P] * 20 + [ctypes.c_size_t, P], ctypes.c_int),
            ("cbr_fp8_quantize", [U] + [P] * 4, ctypes.c_int),
            ("cbr_gemm_fp8_workspace_bytes", [G], ctypes.c_size_t),
            ("cbr_gemm_fp8", [G] + [P] * 7 + [ctypes.c_size_t, P], ctypes.c_int)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = res
    _lib = lib
    return lib


def make_shape(n, h, w, c, k, r, s, stride=1, pad=0, stride_w=None, pad_w=None) -> CbrShape:
    return CbrShape(n, h, w, c, k, r, s, stride, stride if stride_w is None else stride_w,
                    pad, pad if pad_w is None else pad_w)


def _sp(shape):
    return ctypes.byref(shape)


_E_VALUE = 7   # CBR_E_VALUE: the binding reports unusable tensors with it


def _ptr(t, itemsize, name, where, numel=None):
    """Device address of tensor t, after checking that the library can read it as the
    dense array of itemsize-byte elements that include/cbr.h describes: a CUDA (HIP)
    tensor, contiguous in its own layout, with that element size and at least numel
    elements (the count the call's shape implies, when known).  An integer is taken as a
    raw device address; None stays NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise CbrError(_E_VALUE, where, f"{name} is not a GPU tensor")
    if not t.is_contiguous():
        raise CbrError(_E_VALUE, where, f"{name} is not contiguous (the library reads dense NHWC/KRSC arrays)")
    if t.element_size() != itemsize:
        raise CbrError(_E_VALUE, where, f"{name} has {t.element_size()}-byte elements, expected {itemsize}")
    if numel is not None and t.numel() < numel:
        raise CbrError(_E_VALUE, where, f"{name} holds {t.numel()} elements, the shape needs {numel}")
    return t.data_ptr()


def _extents(shape):
    """Element counts of a call's arrays for shape: x (NHWC), w (KRSC), out (NPQK: z, y,
    dy, dz), k (per-channel vectors), mask (32-bit words).  All None when the library
    rejects the shape: it then reports the shape's own error."""
    p, q = ctypes.c_int32(), ctypes.c_int32()
    if _load().cbr_output_hw(_sp(shape), ctypes.byref(p), ctypes.byref(q)) != 0:
        return dict.fromkeys(("x", "w", "out", "k", "mask"))
    s = shape
    return dict(x=s.n * s.h * s.w * s.c, w=s.k * s.r * s.s * s.c, out=s.n * p.value * q.value * s.k, k=s.k,
                mask=cbr_mask_words(shape))


def _ws(workspace, where):
    if workspace is None:
        return None, 0
    if isinstance(workspace, tuple):
        return workspace
    p = _ptr(workspace, workspace.element_size(), "workspace", where)
    return p, workspace.numel() * workspace.element_size()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status, where):
    if status != 0:
        raise CbrError(status, where)


def cbr_status_str(status: int) -> str:
    return _load().cbr_status_str(int(status)).decode()


def cbr_output_hw(shape: CbrShape):
    p, q = ctypes.c_int32(), ctypes.c_int32()
    _check(_load().cbr_output_hw(_sp(shape), ctypes.byref(p), ctypes.byref(q)), "cbr_output_hw")
    return p.value, q.value


def cbr_mask_words(shape: CbrShape) -> int:
    return int(_load().cbr_mask_words(_sp(shape)))


def cbr_workspace_bytes(shape: CbrShape, op: int) -> int:
    return int(_load().cbr_workspace_bytes(_sp(shape), int(op)))


def _events(events):
    """A ctypes array of hipEvent_t handles (torch.cuda.Event objects or raw ints)."""
    if events is None:
        return None
    handles = [e if isinstance(e, int) else e.cuda_event for e in events]
    return (ctypes.c_void_p * len(handles))(*handles)


def cbr_forward_train(shape, x, w, gamma, beta, run_mean_in, run_var_in, eps, momentum,
                      z, y, relu_mask, saved_mean, saved_invstd, run_mean_out, run_var_out,
                      workspace, stream=None, events=None):
    f = "cbr_forward_train"
    ws, nbytes = _ws(workspace, f)
    e = _extents(shape)
    args = (_sp(shape), _ptr(x, 2, "x", f, e["x"]), _ptr(w, 2, "w", f, e["w"]), _ptr(gamma, 4, "gamma", f, e["k"]),
            _ptr(beta, 4, "beta", f, e["k"]), _ptr(run_mean_in, 4, "run_mean_in", f, e["k"]),
            _ptr(run_var_in, 4, "run_var_in", f, e["k"]), float(eps), float(momentum), _ptr(z, 2, "z", f, e["out"]),
            _ptr(y, 2, "y", f, e["out"]), _ptr(relu_mask, 4, "relu_mask", f, e["mask"]),
            _ptr(saved_mean, 4, "saved_mean", f, e["k"]), _ptr(saved_invstd, 4, "saved_invstd", f, e["k"]),
            _ptr(run_mean_out, 4, "run_mean_out", f, e["k"]), _ptr(run_var_out, 4, "run_var_out", f, e["k"]),
            ws, nbytes, _stream(stream))
    if events is None:
        _check(_load().cbr_forward_train(*args), f)
    else:
        _check(_load().cbr_forward_train_ev(*args, _events(events)), "cbr_forward_train_ev")


def cbr_forward_train_noalloc(shape, x, w, gamma, beta, run_mean_in, run_var_in, eps, momentum,
                              z, y, relu_mask, saved_mean, saved_invstd, run_mean_out, run_var_out, stream=None):
    f = "cbr_forward_train_noalloc"
    e = _extents(shape)
    args = (_sp(shape), _ptr(x, 2, "x", f, e["x"]), _ptr(w, 2, "w", f, e["w"]), _ptr(gamma, 4, "gamma", f, e["k"]),
            _ptr(beta, 4, "beta", f, e["k"]), _ptr(run_mean_in, 4, "run_mean_in", f, e["k"]),
            _ptr(run_var_in, 4, "run_var_in", f, e["k"]), float(eps), float(momentum), _ptr(z, 2, "z", f, e["out"]),
            _ptr(y, 2, "y", f, e["out"]), _ptr(relu_mask, 4, "relu_mask", f, e["mask"]),
            _ptr(saved_mean, 4, "saved_mean", f, e["k"]), _ptr(saved_invstd, 4, "saved_invstd", f, e["k"]),
            _ptr(run_mean_out, 4, "run_mean_out", f, e["k"]), _ptr(run_var_out, 4, "run_var_out", f, e["k"]),
            _stream(stream))
    _check(_load().cbr_forward_train_noalloc(*args), f)


def cbr_forward_infer(shape, x, w, conv_bias, gamma, beta, run_mean, run_var, eps, y,
                      workspace, stream=None, events=None):
    f = "cbr_forward_infer"
    ws, nbytes = _ws(workspace, f)
    e = _extents(shape)
    args = (_sp(shape), _ptr(x, 2, "x", f, e["x"]), _ptr(w, 2, "w", f, e["w"]),
            _ptr(conv_bias, 4, "conv_bias", f, e["k"]), _ptr(gamma, 4, "gamma", f, e["k"]),
            _ptr(beta, 4, "beta", f, e["k"]), _ptr(run_mean, 4, "run_mean", f, e["k"]),
            _ptr(run_var, 4, "run_var", f, e["k"]), float(eps), _ptr(y, 2, "y", f, e["out"]), ws, nbytes,
            _stream(stream))
    if events is None:
        _check(_load().cbr_forward_infer(*args), f)
    else:
        _check(_load().cbr_forward_infer_ev(*args, _events(events)), "cbr_forward_infer_ev")


def cbr_backward(shape, x, w, z, relu_mask, dy, gamma, saved_mean, saved_invstd,
                 dz, dgamma, dbeta, dw, dx, workspace, stream=None, events=None):
    f = "cbr_backward"
    ws, nbytes = _ws(workspace, f)
    e = _extents(shape)
    args = (_sp(shape), _ptr(x, 2, "x", f, e["x"]), _ptr(w, 2, "w", f, e["w"]), _ptr(z, 2, "z", f, e["out"]),
            _ptr(relu_mask, 4, "relu_mask", f, e["mask"]), _ptr(dy, 2, "dy", f, e["out"]),
            _ptr(gamma, 4, "gamma", f, e["k"]), _ptr(saved_mean, 4, "saved_mean", f, e["k"]),
            _ptr(saved_invstd, 4, "saved_invstd", f, e["k"]), _ptr(dz, 2, "dz", f, e["out"]),
            _ptr(dgamma, 4, "dgamma", f, e["k"]), _ptr(dbeta, 4, "dbeta", f, e["k"]), _ptr(dw, 4, "dw", f, e["w"]),
            _ptr(dx, 2, "dx", f, e["x"]), ws, nbytes, _stream(stream))
    if events is None:
        _check(_load().cbr_backward(*args), f)
    else:
        _check(_load().cbr_backward_ev(*args, _events(events)), "cbr_backward_ev")


def _conv_bias(name, shape, x, w, bias, y, stream, events):
    e = _extents(shape)
    args = (_sp(shape), _ptr(x, 2, "x", name, e["x"]), _ptr(w, 2, "w", name, e["w"]),
            _ptr(bias, 4, "bias", name, e["k"]), _ptr(y, 2, "y", name, e["out"]), _stream(stream))
    if events is None:
        _check(getattr(_load(), name)(*args), name)
    else:
        _check(getattr(_load(), name + "_ev")(*args, _events(events)), name + "_ev")


def cbr_conv2d_bias_relu(shape, x, w, bias, y, stream=None, events=None):
    _conv_bias("cbr_conv2d_bias_relu", shape, x, w, bias, y, stream, events)


def cbr_conv2d_bias(shape, x, w, bias, y, stream=None, events=None):
    _conv_bias("cbr_conv2d_bias", shape, x, w, bias, y, stream, events)


# Element types that a tensor of each cbr_dtype may have: its own, or an integer of its size.
_DTYPES = {CBR_BF16: ("bfloat16", "int16", "uint16"), CBR_F16: ("float16", "int16", "uint16"),
           CBR_F32: ("float32",), CBR_E4M3: ("float8_e4m3fn", "uint8", "int8"),
           CBR_E5M2: ("float8_e5m2", "uint8", "int8")}


class _Call:
    """One call's view of its tensors: the current device (the one whose stream it runs on) and
    the checks.  These run for every tensor of every call, a dozen of them beside a kernel of a
    few microseconds, so the accepted case is one line; only a refused tensor is looked at
    again to say why."""
    types = None   # cbr_dtype -> frozenset of torch types, made on the first call with `torch`
    torch = None
    __slots__ = ("where", "dev")

    def __init__(self, where, *kinds):
        if _Call.types is None:
            import torch
            _Call.torch = torch
            _Call.types = {k: frozenset(getattr(torch, n) for n in v) for k, v in _DTYPES.items()}
        for k in kinds:
            if k not in _BYTES:
                raise CbrError(_E_VALUE, where)
        self.where = where
        cuda = _Call.torch.cuda
        self.dev = _Call.torch._C._cuda_getDevice() if cuda.is_initialized() else -2

    def at(self, t, kind, name, numel):
        """Device address of tensor t of cbr_dtype kind with numel elements at least (None: not
        known).  None stays NULL, an integer is taken as an address."""
        if t is None:
            return None
        if type(t) is int:
            return t
        if (t.dtype in _Call.types[kind] and t.get_device() == self.dev and t.is_contiguous()
                and (numel is None or t.numel() >= numel)):
            return t.data_ptr()
        p = _ptr(t, _BYTES[kind], name, self.where, numel)
        if t.dtype not in _Call.types[kind]:
            raise CbrError(_E_VALUE, self.where, f"{name} is {t.dtype}, expected torch.{_DTYPES[kind][0]}")
        if t.get_device() != self.torch.cuda.current_device():
            raise CbrError(_E_VALUE, self.where, f"{name} is on GPU {t.get_device()}, the current one is "
                                                 f"{self.torch.cuda.current_device()}")
        return p

    def stream(self, stream):
        """The stream's handle (None: the current one, without the Stream object that
        torch.cuda.current_stream() makes: 2.8 us a call against 0.1)."""
        if stream is None:
            dev = self.dev if self.dev >= 0 else self.torch.cuda.current_device()
            return self.torch._C._cuda_getCurrentRawStream(dev)
        return _stream(stream)

    def workspace(self, workspace):
        """Address and bytes of a workspace (None: none; a pair is taken as they are)."""
        if workspace is None or isinstance(workspace, tuple):
            return _ws(workspace, self.where)
        if workspace.is_cuda and workspace.get_device() != self.torch.cuda.current_device():
            raise CbrError(_E_VALUE, self.where, "workspace is not on the current GPU")
        return _ws(workspace, self.where)


def make_block_shape(rows, channels, rows_per_gate=0, post=CBR_NORM_NONE, pre=CBR_NORM_NONE, stream_type=CBR_BF16,
                     branch_type=CBR_BF16, alpha=1.0, eps_post=1e-5, eps_pre=1e-5) -> CbrBlockShape:
    return CbrBlockShape(rows, rows_per_gate, channels, post, pre, stream_type, branch_type, alpha, eps_post, eps_pre)


def cbr_block_norm_workspace_bytes(shape: CbrBlockShape) -> int:
    return int(_load().cbr_block_norm_workspace_bytes(_sp(shape)))


def cbr_block_norm_forward(shape, x, f, post_w, post_b, gate, res_scale, pre_w, pre_b, y, h, post_stats=None,
                           pre_stats=None, stream=None):
    """y = x + alpha * res_scale * gate * post(f) and h = pre(y), as include/cbr.h describes;
    None is a pointer that is not given."""
    s = shape
    S, B, F = s.stream_type, s.branch_type, CBR_F32
    call = _Call("cbr_block_norm_forward", S, B)
    at, c = call.at, s.channels
    n, st = s.rows * c, 2 * s.rows
    g = s.rows // s.rows_per_gate * c if s.rows_per_gate > 0 else None
    _check(_load().cbr_block_norm_forward(
        _sp(s), at(x, S, "x", n), at(f, B, "f", n), at(post_w, F, "post_w", c), at(post_b, F, "post_b", c),
        at(gate, B, "gate", g), at(res_scale, F, "res_scale", c), at(pre_w, F, "pre_w", c), at(pre_b, F, "pre_b", c),
        at(y, S, "y", n), at(h, B, "h", n), at(post_stats, F, "post_stats", st), at(pre_stats, F, "pre_stats", st),
        call.stream(stream)), call.where)


def cbr_block_norm_backward(shape, dy, dh, y, f, post_w, post_b, gate, res_scale, pre_w, post_stats, pre_stats, dx, df,
                            dpost_w, dpost_b, dgate, dres_scale, dpre_w, dpre_b, workspace, stream=None):
    """Gradients of cbr_block_norm_forward; None is a pointer that is not given (a gradient
    that is not wanted)."""
    s = shape
    S, B, F = s.stream_type, s.branch_type, CBR_F32
    call = _Call("cbr_block_norm_backward", S, B)
    at, c = call.at, s.channels
    n, st = s.rows * c, 2 * s.rows
    g = s.rows // s.rows_per_gate * c if s.rows_per_gate > 0 else None
    ws, nbytes = call.workspace(workspace)
    _check(_load().cbr_block_norm_backward(
        _sp(s), at(dy, S, "dy", n), at(dh, B, "dh", n), at(y, S, "y", n), at(f, B, "f", n), at(post_w, F, "post_w", c),
        at(post_b, F, "post_b", c), at(gate, B, "gate", g), at(res_scale, F, "res_scale", c), at(pre_w, F, "pre_w", c),
        at(post_stats, F, "post_stats", st), at(pre_stats, F, "pre_stats", st), at(dx, S, "dx", n), at(df, B, "df", n),
        at(dpost_w, F, "dpost_w", c), at(dpost_b, F, "dpost_b", c), at(dgate, B, "dgate", g),
        at(dres_scale, F, "dres_scale", c), at(dpre_w, F, "dpre_w", c), at(dpre_b, F, "dpre_b", c), ws, nbytes,
        call.stream(stream)), call.where)


def make_quant_shape(rows, cols, src_type=CBR_BF16, q_type=CBR_E4M3, transpose=False, block=1,
                     ldq=None) -> CbrQuantShape:
    """ldq None: the row length rounded up to 16 bytes."""
    if ldq is None:
        ldq = -(-(rows if transpose else cols) // 16) * 16
    return CbrQuantShape(rows, cols, ldq, src_type, q_type, int(bool(transpose)), block)


def cbr_fp8_quantize(shape, src, q, scale, stream=None):
    """src (or its transpose) in 8 bits, q [rows][ldq] bytes, with its scales (include/cbr.h)."""
    s = shape
    call = _Call("cbr_fp8_quantize", s.src_type, s.q_type)
    if s.block not in (1, 128):
        raise CbrError(_E_VALUE, call.where)
    rows, cols = (s.cols, s.rows) if s.transpose else (s.rows, s.cols)
    _check(_load().cbr_fp8_quantize(_sp(s), call.at(src, s.src_type, "src", s.rows * s.cols),
                                    call.at(q, s.q_type, "q", (rows - 1) * s.ldq + cols),
                                    call.at(scale, CBR_F32, "scale", -(-cols // 128) * -(-rows // s.block)),
                                    call.stream(stream)), call.where)


def make_gemm_shape(m, n, k, a_type=CBR_E4M3, b_type=CBR_E4M3, d_type=CBR_BF16, b_block=128, relu=False, lda=None,
                    ldb=None, short_sums=False) -> CbrGemmShape:
    """lda, ldb None: k rounded up to 16 bytes.  short_sums (16-bit outputs): twice the rate, with sums
    of eight products in 13 bits where the 8-bit matrix instruction is used (include/cbr.h)."""
    ld = -(-k // 16) * 16
    return CbrGemmShape(m, n, k, ld if lda is None else lda, ld if ldb is None else ldb, a_type, b_type, d_type,
                        b_block, int(bool(relu)), int(bool(short_sums)))


def cbr_gemm_fp8_workspace_bytes(shape: CbrGemmShape) -> int:
    return int(_load().cbr_gemm_fp8_workspace_bytes(_sp(shape)))


def cbr_gemm_fp8(shape, a, a_scale, b, b_scale, bias, d, workspace=None, stream=None):
    """d = act((a * a_scale) (b * b_scale)^T + bias) of 8-bit operands (include/cbr.h); workspace
    may be None where cbr_gemm_fp8_workspace_bytes is 0."""
    s = shape
    call = _Call("cbr_gemm_fp8", s.a_type, s.b_type, s.d_type)
    if s.b_block not in (1, 128):
        raise CbrError(_E_VALUE, call.where)
    m, n, kb, at = s.m, s.n, -(-s.k // 128), call.at
    ws, nbytes = call.workspace(workspace)
    _check(_load().cbr_gemm_fp8(_sp(s), at(a, s.a_type, "a", m * s.lda), at(a_scale, CBR_F32, "a_scale", kb * m),
                                at(b, s.b_type, "b", n * s.ldb),
                                at(b_scale, CBR_F32, "b_scale", kb * -(-n // s.b_block)),
                                at(bias, CBR_F32, "bias", n), at(d, s.d_type, "d", m * n), ws, nbytes,
                                call.stream(stream)), call.where)
