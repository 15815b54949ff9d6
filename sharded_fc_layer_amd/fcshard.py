"""Thin Python binding of libfcshard.so (the C ABI declared in include/fcshard.h).

Argument marshalling only: every product runs in the library's HIP kernels.
PyTorch supplies device memory (torch.Tensor) and the current HIP stream.
If the library is not built, every call raises: there is no fallback.

Storage conventions follow the ABI: X is M x K and W is K x N as logical
matrices, each stored row-major (ROW) or column-major (COL); a COL matrix is
passed as the tensor of its transpose (e.g. nn.Linear.weight, N x K, is W in
COL). dY, Y, dX and dW are row-major.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import List, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfcshard.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "fcshard.h")

ROW, COL = 0, 1                # fc_order
OUT_BF16, OUT_F32, OUT_F32_ACC = 0, 1, 2  # fc_out_dtype (OUT_F32_ACC: fp32 out += product)
OP_FWD, OP_BWD_DATA, OP_BWD_WEIGHT = 0, 1, 2  # fc_op
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4  # fc_act
FC_OK, FC_E_INVALID, FC_E_UNSUPPORTED, FC_E_HIP, FC_E_NOMEM, FC_E_TOO_LARGE = 0, 1, 2, 3, 4, 5

_lib = None


class MfmaProbeResult(ctypes.Structure):
    """fc_mfma_probe_result of include/fcshard.h."""
    _fields_ = [("ms", ctypes.c_double), ("flops", ctypes.c_double), ("compute_units", ctypes.c_int),
                ("counter_ratio", ctypes.c_double), ("wall_clock_mhz", ctypes.c_double)]


class FcError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)}")
        self.status = status


def header_functions() -> List[str]:
    """Names of the functions that include/fcshard.h declares."""
    text = open(HEADER).read()
    return re.findall(r"^\s*(?:fc_status|int|int64_t|const char\*)\s+(fc_\w+)\s*\(", text, re.M)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sharded_fc_layer_amd.build`")
        # torch carries its own HIP runtime. Loaded first, it also serves this
        # library's HIP dependency, so torch's memory and streams and this
        # library's calls live in one runtime; loaded after, the process would
        # hold two runtimes and this library's calls fail.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, ci, cs = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.fc_fwd.argtypes = [vp, ci, vp, ci, vp, ci, i64, i64, i64, vp]
        L.fc_bwd_data.argtypes = [vp, vp, ci, vp, ci, i64, i64, i64, vp]
        L.fc_bwd_weight.argtypes = [vp, ci, vp, vp, ci, i64, i64, i64, vp]
        L.fc_bwd_weight_noalloc.argtypes = [vp, ci, vp, vp, ci, i64, i64, i64, vp]
        L.fc_noalloc_scratch_bytes.argtypes = []
        L.fc_noalloc_scratch_bytes.restype = i64
        L.fc_tune.argtypes = [i64, i64, i64, ci, ci, ci, ci, vp]
        L.fc_set_plan.argtypes = [ci, i64, i64, i64, ci, ci, ci, ci]
        L.fc_plan_describe.argtypes = [ci, i64, i64, i64, ci, ci, ci, ctypes.c_char_p, cs]
        L.fc_plan_count.argtypes = []
        L.fc_status_str.argtypes = [ci]
        L.fc_status_str.restype = ctypes.c_char_p
        L.fc_release.argtypes = []
        L.fc_plans_save.argtypes = [ctypes.c_char_p]
        L.fc_plans_load.argtypes = [ctypes.c_char_p]
        L.fc_mfma_probe.argtypes = [i64, ctypes.POINTER(MfmaProbeResult), vp]
        L.fc_mfma_probe_launch.argtypes = [i64, ci, vp, vp]
        L.fc_stamped_call.argtypes = [ci, vp, ci, vp, ci, vp, ci, i64, i64, i64, vp, i64,
                                      ctypes.POINTER(i64), vp]
        L.fc_fwd_act.argtypes = [vp, ci, vp, ci, vp, vp, ci, vp, vp, ci, i64, i64, i64, vp, i64, vp]
        L.fc_bwd_data_act.argtypes = [vp, vp, ci, vp, ci, vp, ci, vp, i64, i64, i64, vp, i64, vp]
        L.fc_bwd_act.argtypes = [vp, vp, ci, vp, vp, i64, i64, vp, i64, vp]
        L.fc_xent_fwd.argtypes = [vp, vp, ci, vp, i64, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp]
        L.fc_xent_bwd.argtypes = [vp, vp, ci, vp, i64, i64, vp, vp, vp, ci, vp, ci, i64, i64, i64, vp, i64, vp]
        L.fc_grouped_fwd.argtypes = [vp, vp, ci, vp, vp, ci, i64, i64, i64, i64, vp, i64, vp]
        L.fc_grouped_bwd_data.argtypes = [vp, vp, ci, vp, vp, ci, i64, i64, i64, i64, vp, i64, vp]
        L.fc_grouped_bwd_weight.argtypes = [vp, vp, vp, vp, ci, i64, i64, i64, i64, vp, i64, vp]
        L.fc_fwd_act_ws_bytes.argtypes = [i64, i64, i64, ci, ci, ci]
        L.fc_bwd_act_ws_bytes.argtypes = [i64, i64]
        L.fc_grouped_ws_bytes.argtypes = [ci, i64, i64, i64, i64, ci, ci]
        for f in (L.fc_bwd_data_act_ws_bytes, L.fc_xent_fwd_ws_bytes, L.fc_xent_bwd_ws_bytes):
            f.argtypes = [i64, i64, i64, ci, ci]
        for f in (L.fc_fwd_act_ws_bytes, L.fc_bwd_data_act_ws_bytes, L.fc_bwd_act_ws_bytes, L.fc_xent_fwd_ws_bytes,
                  L.fc_xent_bwd_ws_bytes, L.fc_grouped_ws_bytes):
            f.restype = i64
        for f in (L.fc_fwd_act, L.fc_bwd_data_act, L.fc_bwd_act, L.fc_xent_fwd, L.fc_xent_bwd, L.fc_grouped_fwd,
                  L.fc_grouped_bwd_data, L.fc_grouped_bwd_weight):
            f.restype = ci
        for f in (L.fc_fwd, L.fc_bwd_data, L.fc_bwd_weight, L.fc_bwd_weight_noalloc, L.fc_tune, L.fc_set_plan, L.fc_plan_describe,
                  L.fc_plan_count, L.fc_release, L.fc_plans_save, L.fc_plans_load, L.fc_mfma_probe,
                  L.fc_mfma_probe_launch, L.fc_stamped_call):
            f.restype = ci
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().fc_status_str(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != FC_OK:
        raise FcError(status, what)


def _stream(stream) -> Optional[int]:
    """A hipStream_t handle: from a torch.cuda.Stream, an int, or torch's current stream."""
    if stream is not None:
        return int(getattr(stream, "cuda_stream", stream))
    import torch
    return torch.cuda.current_stream().cuda_stream


def _bf16_2d(t, name: str):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D torch.bfloat16 tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA/HIP tensor")
    return t


def _logical(t, order: int):
    """(rows, cols) of the logical matrix whose storage is tensor t."""
    r, c = t.shape
    return (r, c) if order == ROW else (c, r)


def _out(out, rows: int, cols: int, out_dtype: int, like, name: str, stream=None):
    """The output tensor: `out` checked, or a new one allocated on the stream that
    writes it (so torch's caching allocator does not hand its memory to other
    work on another stream while the kernels still write it)."""
    import torch
    dt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
    if out is None:
        if out_dtype == OUT_F32_ACC:
            raise ValueError(f"{name}: accumulating needs the existing output tensor (out=)")
        if stream is None or _stream(stream) == torch.cuda.current_stream().cuda_stream:
            return torch.empty((rows, cols), dtype=dt, device=like.device)
        ts = stream if isinstance(stream, torch.cuda.Stream) else \
            torch.cuda.ExternalStream(_stream(stream), device=like.device)
        with torch.cuda.stream(ts):
            return torch.empty((rows, cols), dtype=dt, device=like.device)
    if out.dtype != dt or tuple(out.shape) != (rows, cols) or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {(rows, cols)}")
    if not out.is_cuda:
        raise ValueError(f"{name} must be a CUDA/HIP tensor")
    return out


def _one_device(*ts) -> None:
    """The library runs on the current device: every tensor must live there."""
    import torch
    cur = torch.cuda.current_device()
    for t in ts:
        if t.device.index != cur:
            raise ValueError(f"a tensor is on {t.device}, but the current device is cuda:{cur}")


def fc_fwd(X, W, x_order: int = ROW, w_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """Y = X . W on the GPU; returns Y (M x N, row-major)."""
    _bf16_2d(X, "X"), _bf16_2d(W, "W")
    M, K = _logical(X, x_order)
    K2, N = _logical(W, w_order)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {K2}x{N}")
    Y = _out(out, M, N, out_dtype, X, "out", stream)
    _one_device(X, W, Y)
    _check(lib().fc_fwd(X.data_ptr(), x_order, W.data_ptr(), w_order, Y.data_ptr(), out_dtype, M, K, N,
                        _stream(stream)), "fc_fwd")
    return Y


def fc_bwd_data(dY, W, w_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """dX = dY . W^T on the GPU; returns dX (M x K, row-major)."""
    _bf16_2d(dY, "dY"), _bf16_2d(W, "W")
    M, N = dY.shape
    K, N2 = _logical(W, w_order)
    if N2 != N:
        raise ValueError(f"dY is {M}x{N} but W is {K}x{N2}")
    dX = _out(out, M, K, out_dtype, dY, "out", stream)
    _one_device(dY, W, dX)
    _check(lib().fc_bwd_data(dY.data_ptr(), W.data_ptr(), w_order, dX.data_ptr(), out_dtype, M, K, N,
                             _stream(stream)), "fc_bwd_data")
    return dX


def fc_bwd_weight(X, dY, x_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """dW = X^T . dY on the GPU; returns dW (K x N, row-major)."""
    _bf16_2d(X, "X"), _bf16_2d(dY, "dY")
    M, K = _logical(X, x_order)
    M2, N = dY.shape
    if M2 != M:
        raise ValueError(f"X is {M}x{K} but dY is {M2}x{N}")
    dW = _out(out, K, N, out_dtype, X, "out", stream)
    _one_device(X, dY, dW)
    _check(lib().fc_bwd_weight(X.data_ptr(), x_order, dY.data_ptr(), dW.data_ptr(), out_dtype, M, K, N,
                               _stream(stream)), "fc_bwd_weight")
    return dW


def fc_bwd_weight_noalloc(X, dY, x_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """dW = X^T . dY as fc_bwd_weight, with the plan's staging in the library's
    static device scratch instead of its workspace (the library allocates
    nothing; pass out= for a call that allocates nothing at all)."""
    _bf16_2d(X, "X"), _bf16_2d(dY, "dY")
    M, K = _logical(X, x_order)
    M2, N = dY.shape
    if M2 != M:
        raise ValueError(f"X is {M}x{K} but dY is {M2}x{N}")
    dW = _out(out, K, N, out_dtype, X, "out", stream)
    _one_device(X, dY, dW)
    _check(lib().fc_bwd_weight_noalloc(X.data_ptr(), x_order, dY.data_ptr(), dW.data_ptr(), out_dtype, M, K, N,
                                       _stream(stream)), "fc_bwd_weight_noalloc")
    return dW


# ---- fused operators: activations in the epilogue, the vocabulary's loss, expert layers

class _On:
    """The stream of a call: its handle, and where its tensors are allocated
    (on that stream, so that torch's allocator hands their memory on in its
    order). These calls may take a few microseconds on the GPU, so the host's
    share is kept short: the stream is looked up once."""
    __slots__ = ("handle", "other", "device")

    def __init__(self, stream, like):
        import torch
        self.device = like.device
        if isinstance(stream, torch.cuda.Stream) and stream.device_index != like.get_device():
            raise ValueError(f"the stream is on {stream.device}, the tensors on {like.device}")
        current = torch._C._cuda_getCurrentRawStream(like.get_device() if like.is_cuda else 0)
        self.handle = current if stream is None else _stream(stream)
        self.other = None
        if self.handle != current:
            self.other = stream if isinstance(stream, torch.cuda.Stream) else \
                torch.cuda.ExternalStream(self.handle, device=like.device)

    def empty(self, shape, dtype):
        import torch
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.other):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def given(self, t, dtype, shape, name):
        """An output: the caller's tensor, checked, or a new one."""
        return self.empty(shape, dtype) if t is None else _tensor(t, dtype, shape, name)

    def zero(self, t):
        import torch
        if self.other is None:
            return t.zero_()
        with torch.cuda.stream(self.other):
            return t.zero_()

    def workspace(self, need, what):
        """The call's workspace (None if it needs none), its address and size.
        It may be dropped after the call: its memory is handed on in stream order."""
        if need <= 0:
            if need < 0:
                raise FcError(FC_E_INVALID, what)
            return None, None, 0
        import torch
        ws = self.empty((need,), torch.uint8)
        return ws, ws.data_ptr(), need


def _tensor(t, dtype, shape, name: str):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape:
        raise TypeError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA/HIP tensor")
    return t


def _here(*ts) -> None:
    """The library runs on the current device: every tensor must live there."""
    import torch
    cur = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"a tensor is on {t.device}, but the current device is cuda:{cur}")


def _out_type(out_dtype: int, name: str):
    import torch
    if out_dtype == OUT_BF16:
        return torch.bfloat16
    if out_dtype != OUT_F32:
        raise ValueError(f"{name} must be OUT_BF16 or OUT_F32")
    return torch.float32


def _aligned(a, b) -> int:
    return int((a.data_ptr() | b.data_ptr()) % 16 == 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _order(order: int, name: str) -> int:
    if order != ROW and order != COL:
        raise ValueError(f"{name} must be ROW or COL")
    return order


def fc_fwd_act(X, W, bias=None, act: int = ACT_NONE, residual=None, x_order: int = ROW, w_order: int = ROW,
               keep_z: bool = False, out=None, out_dtype: int = OUT_BF16, z_out=None, stream=None):
    """Y = act(X . W + bias) + residual on the GPU; returns Y (M x N), or (Y, Z)
    with the pre-activation Z (bf16) if keep_z or z_out is given. bias: N bf16
    values; residual: M x N bf16."""
    import torch
    _bf16_2d(X, "X"), _bf16_2d(W, "W"), _order(x_order, "x_order"), _order(w_order, "w_order")
    M, K = _logical(X, x_order)
    K2, N = _logical(W, w_order)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {K2}x{N}")
    if bias is not None:
        _tensor(bias, torch.bfloat16, (N,), "bias")
    if residual is not None:
        _tensor(residual, torch.bfloat16, (M, N), "residual")
    on = _On(stream, X)
    Y = on.given(out, _out_type(out_dtype, "out_dtype"), (M, N), "out")
    Z = on.given(z_out, torch.bfloat16, (M, N), "z_out") if keep_z or z_out is not None else None
    _here(X, W, bias, residual, Y, Z)
    L = lib()
    ws, wp, wn = on.workspace(L.fc_fwd_act_ws_bytes(M, K, N, x_order, w_order, _aligned(X, W)), "fc_fwd_act")
    _check(L.fc_fwd_act(X.data_ptr(), x_order, W.data_ptr(), w_order, _ptr(bias), _ptr(residual), act, _ptr(Z),
                        Y.data_ptr(), out_dtype, M, K, N, wp, wn, on.handle), "fc_fwd_act")
    return Y if Z is None else (Y, Z)


def fc_bwd_data_act(dY, W, Z, act: int, w_order: int = ROW, bias_grad: bool = False, out=None,
                    out_dtype: int = OUT_BF16, db=None, stream=None):
    """dX = (dY . W^T) * act'(Z) on the GPU, Z (M x K, bf16) the pre-activation
    of the layer below; returns dX (M x K), or (dX, db) with the sums of its
    columns (fp32, K values: that layer's bias gradient) if bias_grad or db."""
    import torch
    _bf16_2d(dY, "dY"), _bf16_2d(W, "W"), _order(w_order, "w_order")
    M, N = dY.shape
    K, N2 = _logical(W, w_order)
    if N2 != N:
        raise ValueError(f"dY is {M}x{N} but W is {K}x{N2}")
    _tensor(Z, torch.bfloat16, (M, K), "Z")
    on = _On(stream, dY)
    dX = on.given(out, _out_type(out_dtype, "out_dtype"), (M, K), "out")
    if bias_grad or db is not None:
        db = on.given(db, torch.float32, (K,), "db")
    _here(dY, W, Z, dX, db)
    L = lib()
    ws, wp, wn = on.workspace(L.fc_bwd_data_act_ws_bytes(M, K, N, w_order, _aligned(dY, W)), "fc_bwd_data_act")
    _check(L.fc_bwd_data_act(dY.data_ptr(), W.data_ptr(), w_order, Z.data_ptr(), act, dX.data_ptr(), out_dtype,
                             _ptr(db), M, K, N, wp, wn, on.handle), "fc_bwd_data_act")
    return dX if db is None else (dX, db)


def fc_bwd_act(dY, Z=None, act: int = ACT_NONE, bias_grad: bool = True, keep_dz: bool = True, out=None, db=None,
               stream=None):
    """dZ = dY * act'(Z) and db = the sums of its columns (fp32) on the GPU: the
    first step back through an fc_fwd_act. Returns (dZ, db), None for what was
    not asked for (keep_dz, bias_grad)."""
    import torch
    _bf16_2d(dY, "dY")
    M, N = dY.shape
    if Z is not None:
        _tensor(Z, torch.bfloat16, (M, N), "Z")
    on = _On(stream, dY)
    dZ = on.given(out, torch.bfloat16, (M, N), "out") if keep_dz or out is not None else None
    if bias_grad or db is not None:
        db = on.given(db, torch.float32, (N,), "db")
    _here(dY, Z, dZ, db)
    L = lib()
    ws, wp, wn = on.workspace(L.fc_bwd_act_ws_bytes(M, N) if db is not None else 0, "fc_bwd_act")
    _check(L.fc_bwd_act(dY.data_ptr(), _ptr(Z), act, _ptr(dZ), _ptr(db), M, N, wp, wn, on.handle), "fc_bwd_act")
    return dZ, db


def _xent_operands(X, W, targets, w_order: int):
    import torch
    _bf16_2d(X, "X"), _bf16_2d(W, "W"), _order(w_order, "w_order")
    M, K = X.shape
    K2, N = _logical(W, w_order)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {K2}x{N}")
    _tensor(targets, torch.int64, (M,), "targets")
    return M, K, N


def fc_xent_fwd(X, W, targets, w_order: int = ROW, vocab_start: int = 0, ignore_index: int = -100, stream=None):
    """Cross entropy of the vocabulary projection X . W, without its logits:
    returns (loss, lse, tlogit), M fp32 values each (see fcshard.h; W may be
    the shard of a vocabulary that starts at vocab_start)."""
    import torch
    M, K, N = _xent_operands(X, W, targets, w_order)
    on = _On(stream, X)
    loss, lse, tlogit = (on.empty((M,), torch.float32) for _ in range(3))
    _here(X, W, targets, loss)
    L = lib()
    ws, wp, wn = on.workspace(L.fc_xent_fwd_ws_bytes(M, K, N, w_order, _aligned(X, W)), "fc_xent_fwd")
    _check(L.fc_xent_fwd(X.data_ptr(), W.data_ptr(), w_order, targets.data_ptr(), vocab_start, ignore_index,
                         lse.data_ptr(), tlogit.data_ptr(), loss.data_ptr(), M, K, N, wp, wn, on.handle),
           "fc_xent_fwd")
    return loss, lse, tlogit


def fc_xent_bwd(X, W, targets, lse, grad, w_order: int = ROW, vocab_start: int = 0, ignore_index: int = -100,
                dX=None, dx_dtype: int = OUT_BF16, dW=None, dw_dtype: int = OUT_BF16, stream=None):
    """Gradients of fc_xent_fwd's loss: grad (fp32, M) weighs the rows, lse is
    over the whole vocabulary. Returns (dX, dW): M x K, and K x N row-major;
    dw_dtype = OUT_F32_ACC adds to the given dW."""
    import torch
    M, K, N = _xent_operands(X, W, targets, w_order)
    _tensor(lse, torch.float32, (M,), "lse"), _tensor(grad, torch.float32, (M,), "grad")
    on = _On(stream, X)
    dX = on.given(dX, _out_type(dx_dtype, "dx_dtype"), (M, K), "dX")
    dW = _weight_grad(on, dW, dw_dtype, (K, N), "dW")
    _here(X, W, targets, lse, grad, dX, dW)
    L = lib()
    ws, wp, wn = on.workspace(L.fc_xent_bwd_ws_bytes(M, K, N, w_order, _aligned(X, W)), "fc_xent_bwd")
    _check(L.fc_xent_bwd(X.data_ptr(), W.data_ptr(), w_order, targets.data_ptr(), vocab_start, ignore_index,
                         lse.data_ptr(), grad.data_ptr(), dX.data_ptr(), dx_dtype, dW.data_ptr(), dw_dtype,
                         M, K, N, wp, wn, on.handle), "fc_xent_bwd")
    return dX, dW


def _weight_grad(on, t, dtype: int, shape, name: str):
    """A weight gradient's output of any type; adding to it needs the tensor."""
    import torch
    if dtype == OUT_F32_ACC and t is None:
        raise ValueError(f"{name}: accumulating needs the existing output tensor")
    if dtype == OUT_F32_ACC:
        return _tensor(t, torch.float32, shape, name)
    return on.given(t, _out_type(dtype, name), shape, name)


def _experts(W, w_order: int):
    import torch
    if not isinstance(W, torch.Tensor) or W.dtype != torch.bfloat16 or W.dim() != 3:
        raise TypeError("W must be a 3-D torch.bfloat16 tensor")
    if not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA/HIP tensor")
    _order(w_order, "w_order")
    E, r, c = W.shape
    return (E, r, c) if w_order == ROW else (E, c, r)


def _grouped(op: int, fn, P, Q, offsets, out, out_dtype: int, T: int, E: int, K: int, N: int, w_order: int, on,
             what: str):
    import torch
    _tensor(offsets, torch.int64, (E + 1,), "offsets")
    _here(P, Q, offsets, out)
    if T == 0:  # no row for any expert: the library's sizes start at 1, the answer is known
        if lib().fc_grouped_ws_bytes(op, 1, E, K, N, w_order, 1) < 0:
            raise FcError(FC_E_INVALID, what)
        return on.zero(out) if op == OP_BWD_WEIGHT and out_dtype != OUT_F32_ACC else out
    ws, wp, wn = on.workspace(lib().fc_grouped_ws_bytes(op, T, E, K, N, w_order, _aligned(P, Q)), what)
    orders = () if op == OP_BWD_WEIGHT else (w_order,)
    _check(fn(P.data_ptr(), Q.data_ptr(), *orders, offsets.data_ptr(), out.data_ptr(), out_dtype, T, E, K, N, wp, wn,
              on.handle), what)
    return out


def fc_grouped_fwd(X, W, offsets, w_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """Y = X . W[e] for the rows offsets[e] .. offsets[e + 1] - 1 of each expert
    e: X is T x K, W is E x K x N (COL: E x N x K), offsets E + 1 int64 values
    on the GPU. Rows outside offsets[0] .. offsets[E] of `out` are left as they were.
    T may be 0 in all three calls."""
    _bf16_2d(X, "X")
    E, K, N = _experts(W, w_order)
    T, K2 = X.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: X is {T}x{K2}, W is {K}x{N}")
    on = _On(stream, X)
    Y = on.given(out, _out_type(out_dtype, "out_dtype"), (T, N), "out")
    return _grouped(OP_FWD, lib().fc_grouped_fwd, X, W, offsets, Y, out_dtype, T, E, K, N, w_order, on,
                    "fc_grouped_fwd")


def fc_grouped_bwd_data(dY, W, offsets, w_order: int = ROW, out=None, out_dtype: int = OUT_BF16, stream=None):
    """dX = dY . W[e]^T for each expert's rows (see fc_grouped_fwd)."""
    _bf16_2d(dY, "dY")
    E, K, N = _experts(W, w_order)
    T, N2 = dY.shape
    if N2 != N:
        raise ValueError(f"dY is {T}x{N2} but W is {K}x{N}")
    on = _On(stream, dY)
    dX = on.given(out, _out_type(out_dtype, "out_dtype"), (T, K), "out")
    return _grouped(OP_BWD_DATA, lib().fc_grouped_bwd_data, dY, W, offsets, dX, out_dtype, T, E, K, N, w_order, on,
                    "fc_grouped_bwd_data")


def fc_grouped_bwd_weight(X, dY, offsets, out=None, out_dtype: int = OUT_BF16, stream=None):
    """dW[e] = X^T . dY over each expert's rows: E x K x N, zeros for an expert
    without rows; out_dtype = OUT_F32_ACC adds to the given `out`."""
    import torch
    _bf16_2d(X, "X"), _bf16_2d(dY, "dY")
    T, K = X.shape
    T2, N = dY.shape
    if T2 != T:
        raise ValueError(f"X is {T}x{K} but dY is {T2}x{N}")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise TypeError("offsets must be a torch.int64 tensor of E + 1 values")
    E = offsets.shape[0] - 1
    on = _On(stream, X)
    dW = _weight_grad(on, out, out_dtype, (E, K, N), "out")
    return _grouped(OP_BWD_WEIGHT, lib().fc_grouped_bwd_weight, X, dY, offsets, dW, out_dtype, T, E, K, N, ROW, on,
                    "fc_grouped_bwd_weight")


STAMP_SLOTS = 8  # values per block written by fc_stamped_call


def fc_stamped(op: int, A, B, a_order: int = ROW, b_order: int = ROW, out=None, stamps=None, stream=None):
    """One product with cycle stamps (fc_stamped_call, a measurement aid): the
    same plan and result as the hot call of `op`, with the ring kernel writing
    STAMP_SLOTS counter readings per block.

    op = OP_FWD: A = X (a_order), B = W (b_order); OP_BWD_DATA: A = dY, B = W
    (b_order); OP_BWD_WEIGHT: A = X (a_order), B = dY. The output is bf16.
    Returns (out, stamps): stamps an int64 CUDA tensor (blocks, STAMP_SLOTS),
    laid out as fcshard.h describes. Raises FcError with FC_E_UNSUPPORTED when
    the op's plan has no stamped form (nothing is enqueued then)."""
    import torch
    _bf16_2d(A, "A"), _bf16_2d(B, "B")
    if op == OP_FWD:
        M, K = _logical(A, a_order)
        K2, N = _logical(B, b_order)
        if K2 != K:
            raise ValueError(f"inner dimensions differ: X is {M}x{K}, W is {K2}x{N}")
        rows, cols = M, N
    elif op == OP_BWD_DATA:
        M, N = A.shape
        K, N2 = _logical(B, b_order)
        if N2 != N:
            raise ValueError(f"dY is {M}x{N} but W is {K}x{N2}")
        rows, cols = M, K
    elif op == OP_BWD_WEIGHT:
        M, K = _logical(A, a_order)
        M2, N = B.shape
        if M2 != M:
            raise ValueError(f"X is {M}x{K} but dY is {M2}x{N}")
        rows, cols = K, N
    else:
        raise ValueError(f"unknown op {op}")
    C = _out(out, rows, cols, OUT_BF16, A, "out", stream)
    nb = ((rows + 255) // 256) * ((cols + 255) // 256)
    if stamps is None:
        stamps = torch.zeros((nb, STAMP_SLOTS), dtype=torch.int64, device=A.device)
    if not isinstance(stamps, torch.Tensor) or stamps.dtype != torch.int64 or not stamps.is_cuda \
            or not stamps.is_contiguous() or stamps.dim() != 2 or stamps.shape[1] != STAMP_SLOTS:
        raise ValueError(f"stamps must be a contiguous int64 CUDA tensor of shape (blocks, {STAMP_SLOTS})")
    _one_device(A, B, C, stamps)
    blocks = ctypes.c_int64(0)
    _check(lib().fc_stamped_call(op, A.data_ptr(), a_order, B.data_ptr(), b_order, C.data_ptr(), OUT_BF16,
                                 M, K, N, stamps.data_ptr(), stamps.numel() * 8, ctypes.byref(blocks),
                                 _stream(stream)), "fc_stamped_call")
    return C, stamps[:blocks.value]


def summarize_stamps(stamps, wall_clock_mhz: float, compute_units: Optional[int] = None) -> dict:
    """Per-launch figures from fc_stamped_call's stamps (an integer array of
    shape (blocks, STAMP_SLOTS), on the host): the engine clock while the
    blocks ran (shader-clock ticks over constant-rate ticks), and the mean
    cycles of each block's set-up, prologue (the first stage landing),
    main loop per reduction stage, and epilogue (the output store).

    With compute_units (the stamps of ONE launch), also the launch's span from
    its first block's entry to its last block's exit, in microseconds of the
    constant-rate counter, and the CUs' occupancy: the blocks' summed lifetimes
    over compute_units x that span (one block per CU at a time)."""
    import numpy as np
    s = np.asarray(stamps, dtype=np.float64)
    if s.ndim != 2 or s.shape[1] != STAMP_SLOTS or s.shape[0] == 0:
        raise ValueError(f"stamps must have shape (blocks, {STAMP_SLOTS}), blocks >= 1")
    real = s[:, 6] - s[:, 1]
    if np.any(real <= 0) or np.any(s[:, 7] <= 0):
        raise ValueError("stamps without elapsed time or stages")
    ticks = s[:, 5] - s[:, 0]
    out = {
        "blocks": int(s.shape[0]),
        "clock_GHz": float(ticks.sum() / real.sum() * wall_clock_mhz / 1e3),
        "setup_cycles": float((s[:, 2] - s[:, 0]).mean()),
        "prologue_cycles": float((s[:, 3] - s[:, 2]).mean()),
        "loop_cycles_per_stage": float(((s[:, 4] - s[:, 3]) / s[:, 7]).mean()),
        "epilogue_cycles": float((s[:, 5] - s[:, 4]).mean()),
        "block_cycles": float(ticks.mean()),
        "stages": float(s[:, 7].mean()),
    }
    if compute_units:
        span = float(s[:, 6].max() - s[:, 1].min())
        out["launch_span_us"] = span / wall_clock_mhz
        out["cu_occupancy"] = float(real.sum() / (compute_units * span))
    return out


def fc_noalloc_scratch_bytes() -> int:
    """Size of fc_bwd_weight_noalloc's static device scratch."""
    return int(lib().fc_noalloc_scratch_bytes())


def fc_tune(M: int, K: int, N: int, x_order: int = ROW, w_order: int = ROW, out_dtype: int = OUT_BF16,
            exhaustive: bool = False, warm_caches: bool = False, stream=None) -> None:
    """Time candidate plans of the three products at this shape and cache the fastest
    (with caches flushed before each timed launch unless warm_caches)."""
    flags = (1 if exhaustive else 0) | (2 if warm_caches else 0)
    _check(lib().fc_tune(M, K, N, x_order, w_order, out_dtype, flags, _stream(stream)), "fc_tune")


def fc_plan_count() -> int:
    return int(lib().fc_plan_count())


def fc_set_plan(op: int, M: int, K: int, N: int, x_order: int, w_order: int, out_dtype: int, plan_id: int) -> int:
    """Force a plan (or -1 to clear); returns the status (no raise, for sweeps)."""
    return int(lib().fc_set_plan(op, M, K, N, x_order, w_order, out_dtype, plan_id))


def fc_plan_describe(op: int, M: int, K: int, N: int, x_order: int = ROW, w_order: int = ROW,
                     out_dtype: int = OUT_BF16) -> dict:
    """The plan a hot call would run at this key, parsed into a dict."""
    buf = ctypes.create_string_buffer(512)
    _check(lib().fc_plan_describe(op, M, K, N, x_order, w_order, out_dtype, buf, 512), "fc_plan_describe")
    text = buf.value.decode()
    d = dict(re.findall(r"(\w+)=(gemm_\w+_kernel<[^>]*>|\S+)", text))
    for k in ("plan", "split", "copy", "pad", "ktail", "ws"):
        d[k] = int(d[k])
    if "tuned_ms" in d:
        d["tuned_ms"] = float(d["tuned_ms"])
    return d


def fc_plans_save(path: str) -> None:
    """Write the current device's cached plans to a text file."""
    _check(lib().fc_plans_save(os.fsencode(path)), "fc_plans_save")


def fc_plans_load(path: str) -> None:
    """Load plans saved by fc_plans_save (entries for this device's arch)."""
    _check(lib().fc_plans_load(os.fsencode(path)), "fc_plans_load")


def fc_release() -> None:
    _check(lib().fc_release(), "fc_release")


def fc_mfma_probe(iters: int = 100000, stream=None) -> dict:
    """The MFMA-only stream of the GEMM kernels on every compute unit (measurement
    aid): launch time, flops, compute units and the shader-clock counter ratio."""
    r = MfmaProbeResult()
    _check(lib().fc_mfma_probe(int(iters), ctypes.byref(r), _stream(stream)), "fc_mfma_probe")
    return {"ms": r.ms, "flops": r.flops, "compute_units": r.compute_units, "counter_ratio": r.counter_ratio,
            "wall_clock_mhz": r.wall_clock_mhz}


def fc_mfma_probe_launch(clocks, iters: int = 16, blocks: int = 0, stream=None) -> None:
    """Enqueue the MFMA-only kernel without waiting; block b writes its four
    counter readings to clocks[b] (an int64 CUDA tensor of shape (blocks, 4))."""
    import torch
    if not isinstance(clocks, torch.Tensor) or clocks.dtype != torch.int64 or not clocks.is_cuda \
            or not clocks.is_contiguous() or clocks.dim() != 2 or clocks.shape[1] != 4:
        raise ValueError("clocks must be a contiguous int64 CUDA tensor of shape (blocks, 4)")
    n = clocks.shape[0]
    blocks = int(blocks) or n  # one block per row of clocks by default
    if blocks > n:
        raise ValueError(f"clocks holds {n} blocks, {blocks} requested")
    _one_device(clocks)
    _check(lib().fc_mfma_probe_launch(int(iters), blocks, clocks.data_ptr(), _stream(stream)),
           "fc_mfma_probe_launch")
