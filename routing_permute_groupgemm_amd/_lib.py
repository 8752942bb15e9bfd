"""ctypes binding of libmoe.so (include/moe.h).

Argument marshalling only: torch tensors are checked for dtype/contiguity,
their device pointers and the current HIP stream are passed through, and a
negative status becomes a MoeError.  Every computation runs in the HIP
kernels.  There is no fallback: if the library is missing, loading fails.

stream=: the kernels run on that stream instead of the current one.  The
arguments have to be ready there, and the results, which come from that
stream's memory unless their buffers are given, are ready for the current
stream once it has waited for the other.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

_p = ctypes.c_void_p
_i = ctypes.c_int
_z = ctypes.c_size_t
_i64 = ctypes.c_int64
_f = ctypes.c_float

# every symbol declared in include/moe.h, with its ctypes signature
SIGNATURES = {
    "moe_strerror": ([_i], ctypes.c_char_p),
    "moe_abi_version": ([], _i),
    "moe_route": ([_p, _i, _i, _i, _p, _p, _p], _i),
    "moe_route_backward": ([_p, _p, _p, _i, _i, _i, _p, _p], _i),
    "moe_permute_workspace_size": ([_i, _i, _i], _z),
    "moe_permute": ([_p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _p, _p, _z, _p], _i),
    "moe_permute_noalloc": ([_p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _p, _p], _i),
    "moe_gather": ([_p, _p, _p, _i, _i, _i, _p, _p], _i),
    "moe_gather_gate_grad": ([_p, _p, _p, _p, _i, _i, _i, _p, _p, _p], _i),
    "moe_grouped_gemm_swiglu": ([_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p], _i),
    "moe_grouped_gemm_swiglu_gather": ([_p, _i, _p, _i, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p], _i),
    "moe_grouped_gemm": ([_p, _i, _p, _p, _i, _p, _i, _i, _i, _i, _i, _p, _p, _i, _p], _i),
    "moe_combine": ([_p, _p, _p, _i, _i, _i, _p, _p], _i),
    "moe_wgrad": ([_p, _i, _p, _i, _p, _i, _i, _i, _i, _p, _p], _i),
    "moe_wgrad_gate_up": ([_p, _i, _p, _i, _p, _i, _i, _p, _p, _p], _i),
    "moe_wgrad_gate_up_gather": ([_p, _i, _p, _i, _i, _p, _i, _p, _i, _i, _p, _p, _p], _i),
    "moe_wgrad_split_workspace_size": ([_i, _i, _i, _i], _z),
    "moe_wgrad_split": ([_p, _i, _p, _i, _p, _i, _i, _i, _i, _i, _p, _p, _z, _p], _i),
    "moe_router_workspace_size": ([_i, _i, _i], _z),
    "moe_router_logits": ([_p, _i, _i, _p, _i, _p, _p, _p, _z, _p], _i),
    "moe_router_backward": ([_p, _i, _i, _p, _i, _p, _p, _p, _p, _z, _p], _i),
    "moe_router_bias_backward_workspace_size": ([_i, _i], _z),
    "moe_router_bias_backward": ([_p, _i, _i, _p, _p, _z, _p], _i),
    "moe_pack8": ([_p, _i64, _i, _p, _i, _p, _p, _p], _i),
    "moe_unpack8": ([_p, _p, _i64, _i, _p, _i, _p, _p], _i),
    "moe_grouped_gemm_swiglu_save8": ([_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p], _i),
    "moe_grouped_gemm_swiglu_gather_save8": ([_p, _i, _p, _i, _p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p], _i),
    "moe_grouped_gemm_swiglu_bwd8": ([_p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _p], _i),
    "moe_pack4": ([_p, _i, _i, _i, _p, _p, _p], _i),
    "moe_unpack4": ([_p, _p, _i, _i, _i, _p, _p], _i),
    "moe_grouped_gemm4_swiglu": ([_p, _i, _p, _i, _p, _p, _p, _p, _p, _i, _i, _i, _i, _p, _p], _i),
    "moe_grouped_gemm4": ([_p, _p, _p, _p, _i, _i, _i, _i, _p, _p], _i),
    "moe_gemm4_combine_workspace_size": ([_i, _i], _z),
    "moe_grouped_gemm4_combine": ([_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _i, _i, _p, _p, _p, _z, _p], _i),
    "moe_layer_few_workspace_size": ([_i, _i, _i, _i, _i], _z),
    "moe_layer_few": ([_p, _p, _i, _i, _i, _i, _i, _p, _p, _p, _i, _i, _p, _p, _p, _p, _p, _z, _p], _i),
    "moe_layer_norm": ([_p, _i, _p, _i, _i, _p, _p, _f, _i, _p, _p, _p, _p, _p], _i),
    "moe_layer_norm_backward_workspace_size": ([_i, _i], _z),
    "moe_layer_norm_backward": ([_p, _p, _i, _i, _i, _p, _p, _p, _i, _p, _p, _p, _p, _p, _z, _p], _i),
    "moe_linear_workspace_size": ([_i, _i, _i], _z),
    "moe_linear": ([_p, _i, _i, _p, _i, _p, _i, _p, _p, _p, _p, _z, _p], _i),
    "moe_linear_backward_workspace_size": ([_i, _i, _i], _z),
    "moe_linear_backward": ([_p, _p, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _p, _z, _p], _i),
    "moe_probe_mfma": ([_p, _i, _i, _p, _p], _i),
    "moe_probe_mfma16": ([_p, _i, _i, _p, _p], _i),
    "moe_probe_copy": ([_p, _p, _i64, _i, _i, _p], _i),
}

MOE_EPI_NONE = 0
MOE_EPI_SWIGLU_BWD = 1
MOE_FEW_TOKENS = 64
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}  # moe_act

_lib = None


class MoeError(RuntimeError):
    pass


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() first")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise MoeError(f"libmoe status {status}: {load().moe_strerror(status).decode()}")


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (2.5 us less per call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _empty(shape, dtype, dev, stream, result=True):
    """A new buffer for kernels on this stream (None: the current one).  It comes from that stream's memory: work
    queued earlier on what the memory held, and later allocations once a workspace is dropped at the return, are
    ordered with the kernels.  A result may be read on the current stream, which waits for the other first, so the
    allocator is told of that stream: what is dropped there is not handed out while it is still being read."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if result:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _device(stream, t):
    """The current device, which the stream (None: its current one) must belong to; t: a first argument, refused
    here if it is on the host (there may be no device then)."""
    if not t.is_cuda:
        raise MoeError(f"expected CUDA tensors, got one on {t.device}")
    dev = torch.cuda.current_device()
    if stream is not None and stream.device_index != dev:
        raise MoeError(f"a stream of device {stream.device_index} with device {dev} current")
    return dev


def _arg(t, dtype, name, dev):
    """A contiguous tensor of this type on this device."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise MoeError(f"{name}: expected a contiguous {dtype} tensor on CUDA device {dev}, got {t.dtype} "
                       f"contiguous={t.is_contiguous()} device={t.device}")


def _handle(stream, dev):
    """The stream's handle, dev being the current device."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _need(t, dtype, name):
    if t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise MoeError(f"{name}: expected a contiguous {dtype} CUDA tensor, got {t.dtype} "
                       f"contiguous={t.is_contiguous()} device={t.device}")


def _shape(t, shape, name):
    """A caller-provided buffer must have exactly this shape (the kernels write all of it)."""
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, rows, cols, name):
    """A row buffer of the expert-grouped order: at least `rows` rows of exactly `cols` columns."""
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != cols:
        raise MoeError(f"{name}: expected at least {rows} rows of {cols} columns, got {tuple(t.shape)}")


def moe_route(logits, K, topk_idx=None, gates=None, stream=None):
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    if topk_idx is None:
        topk_idx = _empty((T, K), torch.int32, logits.device, stream)
    if gates is None:
        gates = _empty((T, K), torch.float32, logits.device, stream)
    _need(topk_idx, torch.int32, "topk_idx")
    _need(gates, torch.float32, "gates")
    _shape(topk_idx, (T, K), "topk_idx")
    _shape(gates, (T, K), "gates")
    _check(load().moe_route(_ptr(logits), T, E, K, _ptr(topk_idx), _ptr(gates), _stream(stream)))
    return topk_idx, gates


def moe_route_backward(topk_idx, gates, dgates, E, dlogits=None, stream=None):
    _need(topk_idx, torch.int32, "topk_idx")
    _need(gates, torch.float32, "gates")
    _need(dgates, torch.float32, "dgates")
    T, K = topk_idx.shape
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, gates.device, stream)
    _need(dlogits, torch.float32, "dlogits")
    _shape(gates, (T, K), "gates")
    _shape(dgates, (T, K), "dgates")
    _shape(dlogits, (T, E), "dlogits")
    _check(load().moe_route_backward(_ptr(topk_idx), _ptr(gates), _ptr(dgates), T, E, K, _ptr(dlogits),
                                     _stream(stream)))
    return dlogits


def moe_permute_workspace_size(T, K, e_local) -> int:
    return int(load().moe_permute_workspace_size(T, K, e_local))


def moe_permute(topk_idx, e_begin, e_local, x, cap_rows, out=None, ws=None, stream=None, copy_rows=True):
    """-> dict(counts, offsets, pos, src, x_perm, status) (all device tensors).

    copy_rows=False: the index-only permutation (x_perm is None), for the
    gate/up GroupGEMM that reads x through src."""
    _need(topk_idx, torch.int32, "topk_idx")
    _need(x, torch.bfloat16, "x")
    T, K = topk_idx.shape
    H = x.shape[1]
    dev = x.device
    o = out or {}
    counts = o.get("counts")
    if counts is None:
        counts = _empty(max(e_local, 1), torch.int32, dev, stream)
    offsets = o.get("offsets")
    if offsets is None:
        offsets = _empty(e_local + 1, torch.int32, dev, stream)
    pos = o.get("pos")
    if pos is None:
        pos = _empty((T, K), torch.int32, dev, stream)
    src = o.get("src")
    if src is None:
        src = _empty(max(cap_rows, 1), torch.int32, dev, stream)
    x_perm = o.get("x_perm")
    if x_perm is None and copy_rows:
        x_perm = _empty((max(cap_rows, 1), H), torch.bfloat16, dev, stream)
    if not copy_rows:
        x_perm = None
    status = o.get("status")
    if status is None:
        status = _empty(4, torch.int32, dev, stream)
    need = moe_permute_workspace_size(T, K, e_local)
    if ws is None or ws.numel() < need:
        ws = _empty(max(need, 256), torch.uint8, dev, stream)
    for t, name, dt in ((counts, "counts", torch.int32), (offsets, "offsets", torch.int32), (pos, "pos", torch.int32),
                        (src, "src", torch.int32), (status, "status", torch.int32)):
        _need(t, dt, name)
    if counts.numel() < e_local or offsets.numel() < e_local + 1 or src.numel() < cap_rows or status.numel() < 1:
        raise MoeError("moe_permute: counts, offsets, src or status smaller than e_local, e_local+1, cap_rows, 1")
    _shape(pos, (T, K), "pos")
    if x_perm is not None:
        _need(x_perm, torch.bfloat16, "x_perm")
        _rows(x_perm, cap_rows, H, "x_perm")
    _check(load().moe_permute(_ptr(topk_idx), T, K, e_begin, e_local, _ptr(x), H, cap_rows,
                              _ptr(counts), _ptr(offsets), _ptr(pos), _ptr(src), _ptr(x_perm),
                              _ptr(status), _ptr(ws), ws.numel(), _stream(stream)))
    return dict(counts=counts[:e_local], offsets=offsets, pos=pos, src=src, x_perm=x_perm,
                status=status, ws=ws)


def moe_permute_noalloc(topk_idx, e_begin, e_local, x, cap_rows, out, stream=None, copy_rows=True):
    """moe_permute without a workspace: the library's own device array holds the count matrix.  Every
    output buffer is the caller's (out: counts, offsets, pos, src, status, and x_perm unless
    copy_rows=False); nothing is allocated here either."""
    _need(topk_idx, torch.int32, "topk_idx")
    _need(x, torch.bfloat16, "x")
    T, K = topk_idx.shape
    H = x.shape[1]
    counts, offsets, pos, src, status = (out[k] for k in ("counts", "offsets", "pos", "src", "status"))
    x_perm = out.get("x_perm") if copy_rows else None
    if copy_rows and x_perm is None:
        raise MoeError("moe_permute_noalloc: out['x_perm'] is required with copy_rows=True")
    for t, name, dt in ((counts, "counts", torch.int32), (offsets, "offsets", torch.int32), (pos, "pos", torch.int32),
                        (src, "src", torch.int32), (status, "status", torch.int32)):
        _need(t, dt, name)
    if counts.numel() < e_local or offsets.numel() < e_local + 1 or src.numel() < cap_rows or status.numel() < 1:
        raise MoeError("moe_permute_noalloc: counts, offsets, src or status smaller than e_local, e_local+1, "
                       "cap_rows, 1")
    _shape(pos, (T, K), "pos")
    if x_perm is not None:
        _need(x_perm, torch.bfloat16, "x_perm")
        _rows(x_perm, cap_rows, H, "x_perm")
    _check(load().moe_permute_noalloc(_ptr(topk_idx), T, K, e_begin, e_local, _ptr(x), H, cap_rows,
                                      _ptr(counts), _ptr(offsets), _ptr(pos), _ptr(src), _ptr(x_perm),
                                      _ptr(status), _stream(stream)))
    return dict(counts=counts[:e_local], offsets=offsets, pos=pos, src=src, x_perm=x_perm, status=status)


def moe_gather(d_out, pos, gates, dy_perm, stream=None):
    _need(d_out, torch.bfloat16, "d_out")
    _need(pos, torch.int32, "pos")
    if gates is not None:
        _need(gates, torch.float32, "gates")
    _need(dy_perm, torch.bfloat16, "dy_perm")
    T, K = pos.shape
    _shape(d_out, (T, d_out.shape[1]), "d_out")
    if dy_perm.dim() != 2 or dy_perm.shape[1] != d_out.shape[1]:
        raise MoeError(f"dy_perm: expected rows of {d_out.shape[1]} columns, got {tuple(dy_perm.shape)}")
    if gates is not None:
        _shape(gates, (T, K), "gates")
    _check(load().moe_gather(_ptr(d_out), _ptr(pos), _ptr(gates), T, K, d_out.shape[1], _ptr(dy_perm),
                             _stream(stream)))
    return dy_perm


def moe_gather_gate_grad(d_out, pos, gates, y, dy_perm, dgates=None, stream=None):
    """dy_perm as moe_gather, and dgates[t,k] = <d_out[t], y[pos[t,k]]> (0 for non-local pairs)."""
    _need(d_out, torch.bfloat16, "d_out")
    _need(pos, torch.int32, "pos")
    _need(gates, torch.float32, "gates")
    _need(y, torch.bfloat16, "y")
    _need(dy_perm, torch.bfloat16, "dy_perm")
    T, K = pos.shape
    if dgates is None:
        dgates = _empty((T, K), torch.float32, d_out.device, stream)
    _need(dgates, torch.float32, "dgates")
    H = d_out.shape[1]
    _shape(d_out, (T, H), "d_out")
    _shape(gates, (T, K), "gates")
    _shape(dgates, (T, K), "dgates")
    for t, name in ((y, "y"), (dy_perm, "dy_perm")):
        if t.dim() != 2 or t.shape[1] != H:
            raise MoeError(f"{name}: expected rows of {H} columns, got {tuple(t.shape)}")
    _check(load().moe_gather_gate_grad(_ptr(d_out), _ptr(pos), _ptr(gates), _ptr(y), T, K, d_out.shape[1],
                                       _ptr(dy_perm), _ptr(dgates), _stream(stream)))
    return dy_perm, dgates


def _gate_up_checks(w_gate, w_up, offsets, cap_rows, h, ab_save):
    EL, H, F = w_gate.shape
    _shape(w_up, (EL, H, F), "w_up")
    if offsets.numel() < EL + 1:
        raise MoeError(f"offsets: expected {EL + 1} entries, got {offsets.numel()}")
    _need(h, torch.bfloat16, "h")
    _rows(h, cap_rows, F, "h")
    if ab_save is not None:
        _need(ab_save, torch.bfloat16, "ab_save")
        _rows(ab_save, cap_rows, 2 * F, "ab_save")


def moe_grouped_gemm_swiglu(x_perm, w_gate, w_up, offsets, cap_rows, h=None, ab_save=None, stream=None):
    _need(x_perm, torch.bfloat16, "x_perm")
    _need(w_gate, torch.bfloat16, "w_gate")
    _need(w_up, torch.bfloat16, "w_up")
    _need(offsets, torch.int32, "offsets")
    EL, H, F = w_gate.shape
    if h is None:
        h = _empty((x_perm.shape[0], F), torch.bfloat16, x_perm.device, stream)
    _gate_up_checks(w_gate, w_up, offsets, cap_rows, h, ab_save)
    _rows(x_perm, cap_rows, H, "x_perm")
    _check(load().moe_grouped_gemm_swiglu(_ptr(x_perm), _ptr(w_gate), _ptr(w_up), _ptr(offsets), EL, H, F,
                                          cap_rows, _ptr(h), _ptr(ab_save), _stream(stream)))
    return h


def moe_grouped_gemm_swiglu_gather(x, src, K, w_gate, w_up, offsets, cap_rows, h=None, ab_save=None,
                                   stream=None):
    """Gate/up GroupGEMM + SwiGLU reading row r of the expert-grouped order
    straight from x[src[r] // K] (no x_perm)."""
    _need(x, torch.bfloat16, "x")
    _need(src, torch.int32, "src")
    _need(w_gate, torch.bfloat16, "w_gate")
    _need(w_up, torch.bfloat16, "w_up")
    _need(offsets, torch.int32, "offsets")
    EL, H, F = w_gate.shape
    T = x.shape[0]
    if h is None:
        h = _empty((max(cap_rows, 1), F), torch.bfloat16, x.device, stream)
    _gate_up_checks(w_gate, w_up, offsets, cap_rows, h, ab_save)
    _shape(x, (T, H), "x")
    if src.numel() < cap_rows:
        raise MoeError(f"src: expected at least {cap_rows} entries, got {src.numel()}")
    _check(load().moe_grouped_gemm_swiglu_gather(_ptr(x), T, _ptr(src), int(K), _ptr(w_gate), _ptr(w_up),
                                                 _ptr(offsets), EL, H, F, cap_rows, _ptr(h), _ptr(ab_save),
                                                 _stream(stream)))
    return h


def moe_grouped_gemm(a, w0, w1, trans_w, offsets, Kd, N, cap_rows, c, epilogue=MOE_EPI_NONE, ab=None,
                     lda=None, ldc=None, stream=None):
    _need(a, torch.bfloat16, "a")
    _need(w0, torch.bfloat16, "w0")
    if w1 is not None:
        _need(w1, torch.bfloat16, "w1")
    _need(offsets, torch.int32, "offsets")
    _need(c, torch.bfloat16, "c")
    if ab is not None:
        _need(ab, torch.bfloat16, "ab")
    EL = w0.shape[0]
    lda = a.shape[1] if lda is None else lda
    ldc = c.shape[1] if ldc is None else ldc
    _shape(w0, (EL, N, Kd) if trans_w else (EL, Kd, N), "w0")
    if w1 is not None:
        _shape(w1, tuple(w0.shape), "w1")
    if offsets.numel() < EL + 1:
        raise MoeError(f"offsets: expected {EL + 1} entries, got {offsets.numel()}")
    # every row r < cap_rows of a and c may be touched, at strides lda and ldc
    for t, ld, name in ((a, lda, "a"), (c, ldc, "c")):
        if t.dim() != 2 or t.shape[0] < cap_rows or (cap_rows > 0 and t.shape[1] < ld):
            raise MoeError(f"{name}: expected at least {cap_rows} rows of {ld} columns, got {tuple(t.shape)}")
    if ab is not None:
        _rows(ab, cap_rows, 2 * N, "ab")
    _check(load().moe_grouped_gemm(_ptr(a), lda, _ptr(w0), _ptr(w1), int(trans_w), _ptr(offsets), EL, Kd, N,
                                   cap_rows, epilogue, _ptr(ab), _ptr(c), ldc, _stream(stream)))
    return c


def moe_combine(y, pos, gates, out=None, stream=None):
    _need(y, torch.bfloat16, "y")
    _need(pos, torch.int32, "pos")
    if gates is not None:
        _need(gates, torch.float32, "gates")
    T, K = pos.shape
    H = y.shape[1]
    if out is None:
        out = _empty((T, H), torch.bfloat16, y.device, stream)
    _need(out, torch.bfloat16, "out")
    _shape(out, (T, H), "out")
    if gates is not None:
        _shape(gates, (T, K), "gates")
    _check(load().moe_combine(_ptr(y), _ptr(pos), _ptr(gates), T, K, H, _ptr(out), _stream(stream)))
    return out


def moe_wgrad(a, lda, b, ldb, offsets, e_local, M, N, cap_rows, dw=None, a_col0=0, b_col0=0, stream=None):
    """dw[j] = a_j^T b_j. a_col0/b_col0 offset the first column (e.g. b_col0=F for dW_up from dab)."""
    _need(a, torch.bfloat16, "a")
    _need(b, torch.bfloat16, "b")
    _need(offsets, torch.int32, "offsets")
    if dw is None:
        dw = _empty((e_local, M, N), torch.float32, a.device, stream)
    _need(dw, torch.float32, "dw")
    _shape(dw, (e_local, M, N), "dw")
    if offsets.numel() < e_local + 1:
        raise MoeError(f"offsets: expected {e_local + 1} entries, got {offsets.numel()}")
    # rows r < cap_rows are read at strides lda and ldb from the column offsets
    for t, ld, c0, w, name in ((a, lda, a_col0, M, "a"), (b, ldb, b_col0, N, "b")):
        if cap_rows > 0 and t.numel() < (cap_rows - 1) * ld + c0 + w:
            raise MoeError(f"{name}: too small for {cap_rows} rows at stride {ld} from column {c0}")
    pa = a.data_ptr() + 2 * a_col0
    pb = b.data_ptr() + 2 * b_col0
    _check(load().moe_wgrad(pa, lda, pb, ldb, _ptr(offsets), e_local, M, N, cap_rows, _ptr(dw),
                            _stream(stream)))
    return dw


def moe_wgrad_gate_up(x_perm, dab, offsets, e_local, cap_rows, dw_gate=None, dw_up=None, stream=None):
    """(dw_gate, dw_up) = x_perm_j^T . [da_j | db_j] per expert, in one pass over x_perm."""
    _need(x_perm, torch.bfloat16, "x_perm")
    _need(dab, torch.bfloat16, "dab")
    _need(offsets, torch.int32, "offsets")
    H = x_perm.shape[1]
    F = dab.shape[1] // 2
    if dab.dim() != 2 or dab.shape[1] != 2 * F:
        raise MoeError(f"dab: expected [rows, 2F], got {tuple(dab.shape)}")
    _rows(x_perm, cap_rows, H, "x_perm")
    _rows(dab, cap_rows, 2 * F, "dab")
    if offsets.numel() < e_local + 1:
        raise MoeError(f"offsets: expected {e_local + 1} entries, got {offsets.numel()}")
    out = []
    for t, name in ((dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is None:
            t = _empty((e_local, H, F), torch.float32, x_perm.device, stream)
        _need(t, torch.float32, name)
        _shape(t, (e_local, H, F), name)
        out.append(t)
    _check(load().moe_wgrad_gate_up(_ptr(x_perm), H, _ptr(dab), F, _ptr(offsets), e_local, cap_rows, _ptr(out[0]),
                                    _ptr(out[1]), _stream(stream)))
    return out[0], out[1]


def moe_wgrad_gate_up_gather(x, src, K, dab, offsets, e_local, cap_rows, dw_gate=None, dw_up=None, stream=None):
    """moe_wgrad_gate_up reading row r of the expert-grouped order straight from x[src[r] // K] (no x_perm)."""
    _need(x, torch.bfloat16, "x")
    _need(src, torch.int32, "src")
    _need(dab, torch.bfloat16, "dab")
    _need(offsets, torch.int32, "offsets")
    if x.dim() != 2:
        raise MoeError(f"x: expected [T, H], got {tuple(x.shape)}")
    T, H = x.shape
    F = dab.shape[1] // 2
    if dab.dim() != 2 or dab.shape[1] != 2 * F:
        raise MoeError(f"dab: expected [rows, 2F], got {tuple(dab.shape)}")
    _rows(dab, cap_rows, 2 * F, "dab")
    if src.numel() < cap_rows:
        raise MoeError(f"src: expected at least {cap_rows} entries, got {src.numel()}")
    if offsets.numel() < e_local + 1:
        raise MoeError(f"offsets: expected {e_local + 1} entries, got {offsets.numel()}")
    out = []
    for t, name in ((dw_gate, "dw_gate"), (dw_up, "dw_up")):
        if t is None:
            t = _empty((e_local, H, F), torch.float32, x.device, stream)
        _need(t, torch.float32, name)
        _shape(t, (e_local, H, F), name)
        out.append(t)
    _check(load().moe_wgrad_gate_up_gather(_ptr(x), T, _ptr(src), int(K), H, _ptr(dab), F, _ptr(offsets), e_local,
                                           cap_rows, _ptr(out[0]), _ptr(out[1]), _stream(stream)))
    return out[0], out[1]


def moe_wgrad_split_workspace_size(e_local, M, N, splits) -> int:
    return int(load().moe_wgrad_split_workspace_size(e_local, M, N, splits))


def moe_wgrad_split(a, lda, b, ldb, offsets, e_local, M, N, cap_rows, splits, dw=None, ws=None, a_col0=0,
                    b_col0=0, stream=None):
    """moe_wgrad with each expert's rows in `splits` fixed chunks whose fp32 partials are added in chunk
    order (ws: device workspace, allocated here if not given or too small)."""
    _need(a, torch.bfloat16, "a")
    _need(b, torch.bfloat16, "b")
    _need(offsets, torch.int32, "offsets")
    if dw is None:
        dw = _empty((e_local, M, N), torch.float32, a.device, stream)
    _need(dw, torch.float32, "dw")
    _shape(dw, (e_local, M, N), "dw")
    if offsets.numel() < e_local + 1:
        raise MoeError(f"offsets: expected {e_local + 1} entries, got {offsets.numel()}")
    for t, ld, c0, w, name in ((a, lda, a_col0, M, "a"), (b, ldb, b_col0, N, "b")):
        if cap_rows > 0 and t.numel() < (cap_rows - 1) * ld + c0 + w:
            raise MoeError(f"{name}: too small for {cap_rows} rows at stride {ld} from column {c0}")
    need = moe_wgrad_split_workspace_size(e_local, M, N, splits)
    if ws is None or ws.numel() < need:
        ws = _empty(max(need, 256), torch.uint8, a.device, stream, result=False)
    pa = a.data_ptr() + 2 * a_col0
    pb = b.data_ptr() + 2 * b_col0
    _check(load().moe_wgrad_split(pa, lda, pb, ldb, _ptr(offsets), e_local, M, N, cap_rows, splits, _ptr(dw),
                                  _ptr(ws), ws.numel(), _stream(stream)))
    return dw


def moe_router_workspace_size(T, H, E) -> int:
    return int(load().moe_router_workspace_size(T, H, E))


def _router_ws(T, H, E, ws, dev, stream):
    need = moe_router_workspace_size(T, H, E)
    if ws is None or ws.numel() < need:
        ws = _empty(max(need, 256), torch.uint8, dev, stream, result=False)
    return ws


def moe_router_logits(x, w_r, bias=None, logits=None, ws=None, stream=None):
    """logits fp32 [T,E] = x . w_r (+ bias)."""
    _need(x, torch.bfloat16, "x")
    _need(w_r, torch.bfloat16, "w_r")
    if bias is not None:
        _need(bias, torch.float32, "bias")
    T, H = x.shape
    E = w_r.shape[1]
    if logits is None:
        logits = _empty((T, E), torch.float32, x.device, stream)
    _shape(w_r, (H, E), "w_r")
    if bias is not None:
        _shape(bias, (E,), "bias")
    _need(logits, torch.float32, "logits")
    _shape(logits, (T, E), "logits")
    ws = _router_ws(T, H, E, ws, x.device, stream)
    _check(load().moe_router_logits(_ptr(x), T, H, _ptr(w_r), E, _ptr(bias), _ptr(logits), _ptr(ws), ws.numel(),
                                    _stream(stream)))
    return logits


def moe_router_backward(x, w_r, dlogits, dx=None, dw_r=None, ws=None, stream=None):
    """-> (dx bf16 [T,H], dw_r fp32 [H,E]) of the router projection."""
    _need(x, torch.bfloat16, "x")
    _need(w_r, torch.bfloat16, "w_r")
    _need(dlogits, torch.float32, "dlogits")
    T, H = x.shape
    E = w_r.shape[1]
    if dx is None:
        dx = _empty((T, H), torch.bfloat16, x.device, stream)
    if dw_r is None:
        dw_r = _empty((H, E), torch.float32, x.device, stream)
    _shape(w_r, (H, E), "w_r")
    _shape(dlogits, (T, E), "dlogits")
    _need(dx, torch.bfloat16, "dx")
    _shape(dx, (T, H), "dx")
    _need(dw_r, torch.float32, "dw_r")
    _shape(dw_r, (H, E), "dw_r")
    ws = _router_ws(T, H, E, ws, x.device, stream)
    _check(load().moe_router_backward(_ptr(x), T, H, _ptr(w_r), E, _ptr(dlogits), _ptr(dx), _ptr(dw_r), _ptr(ws),
                                      ws.numel(), _stream(stream)))
    return dx, dw_r


def _routed(offsets, dev):
    """offsets or None -> its expert count (0 without)."""
    if offsets is None:
        return 0
    _arg(offsets, torch.int32, "offsets", dev)
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise MoeError(f"offsets: expected e_local + 1 entries, got {tuple(offsets.shape)}")
    return offsets.numel() - 1


def _offsets(offsets, EL, dev):
    _arg(offsets, torch.int32, "offsets", dev)
    if offsets.numel() < EL + 1:
        raise MoeError(f"offsets: expected {EL + 1} entries, got {offsets.numel()}")


def _out(t, shape, dtype, name, dev, stream, rows=None):
    """The caller's buffer (checked: at least `rows` rows, or exactly `shape`) or a new one."""
    if t is None:
        return _empty(shape, dtype, dev, stream)
    _arg(t, dtype, name, dev)
    if rows is None:
        _shape(t, shape, name)
    else:
        _rows(t, rows, shape[1], name)
    return t


def moe_pack8(x, q=None, scale=None, offsets=None, stream=None):
    """Rows of bf16 -> (q int8 [rows, cols], scale uint8 [rows, cols/32]) in blocks of 32 columns.
    offsets (int32 [e_local+1]): only the first offsets[e_local] rows are read and written."""
    dev = _device(stream, x)
    _arg(x, torch.bfloat16, "x", dev)
    if x.dim() != 2 or x.shape[1] % 64:
        raise MoeError(f"x: expected [rows, a multiple of 64], got {tuple(x.shape)}")
    rows, cols = x.shape
    EL = _routed(offsets, dev)
    q = _out(q, (rows, cols), torch.int8, "q", dev, stream, rows)
    scale = _out(scale, (rows, cols // 32), torch.uint8, "scale", dev, stream, rows)
    _check(load().moe_pack8(_ptr(x), rows, cols, _ptr(offsets), EL, _ptr(q), _ptr(scale), _handle(stream, dev)))
    return q, scale


def moe_unpack8(q, scale, x=None, offsets=None, stream=None):
    """The bf16 rows that (q, scale) stand for (rows and offsets as moe_pack8)."""
    dev = _device(stream, q)
    _arg(q, torch.int8, "q", dev)
    _arg(scale, torch.uint8, "scale", dev)
    if q.dim() != 2 or q.shape[1] % 64:
        raise MoeError(f"q: expected [rows, a multiple of 64], got {tuple(q.shape)}")
    rows, cols = q.shape
    EL = _routed(offsets, dev)
    _rows(scale, rows, cols // 32, "scale")
    x = _out(x, (rows, cols), torch.bfloat16, "x", dev, stream, rows)
    _check(load().moe_unpack8(_ptr(q), _ptr(scale), rows, cols, _ptr(offsets), EL, _ptr(x), _handle(stream, dev)))
    return x


def _save8_args(x, w_gate, w_up, offsets, cap_rows, h, ab8, ab8_scale, dev, stream):
    """Checks common to the two forms -> (EL, H, F, h, ab8, ab8_scale)."""
    for t, name in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up")):
        _arg(t, torch.bfloat16, name, dev)
    if w_gate.dim() != 3:
        raise MoeError(f"w_gate: expected [E, H, F], got {tuple(w_gate.shape)}")
    EL, H, F = w_gate.shape
    _shape(w_up, (EL, H, F), "w_up")
    _offsets(offsets, EL, dev)
    n = max(cap_rows, 0)
    h = _out(h, (n, F), torch.bfloat16, "h", dev, stream, n)
    ab8 = _out(ab8, (n, 2 * F), torch.int8, "ab8", dev, stream, n)
    ab8_scale = _out(ab8_scale, (n, 2 * F // 32), torch.uint8, "ab8_scale", dev, stream, n)
    return EL, H, F, h, ab8, ab8_scale


def moe_grouped_gemm_swiglu_save8(x_perm, w_gate, w_up, offsets, cap_rows, h=None, ab8=None, ab8_scale=None,
                                  stream=None):
    """moe_grouped_gemm_swiglu with (a, b) saved in 8-bit blocks -> (h, ab8, ab8_scale)."""
    dev = _device(stream, x_perm)
    EL, H, F, h, ab8, ab8_scale = _save8_args(x_perm, w_gate, w_up, offsets, cap_rows, h, ab8, ab8_scale, dev,
                                              stream)
    _rows(x_perm, cap_rows, H, "x_perm")
    _check(load().moe_grouped_gemm_swiglu_save8(_ptr(x_perm), _ptr(w_gate), _ptr(w_up), _ptr(offsets), EL, H, F,
                                                cap_rows, _ptr(h), _ptr(ab8), _ptr(ab8_scale), _handle(stream, dev)))
    return h, ab8, ab8_scale


def moe_grouped_gemm_swiglu_gather_save8(x, src, K, w_gate, w_up, offsets, cap_rows, h=None, ab8=None,
                                         ab8_scale=None, stream=None):
    """The same, reading row r of the expert-grouped order from x[src[r] // K] (no x_perm)."""
    dev = _device(stream, x)
    EL, H, F, h, ab8, ab8_scale = _save8_args(x, w_gate, w_up, offsets, cap_rows, h, ab8, ab8_scale, dev, stream)
    _rows(x, 0, H, "x")
    _arg(src, torch.int32, "src", dev)
    if src.numel() < cap_rows:
        raise MoeError(f"src: expected at least {cap_rows} entries, got {src.numel()}")
    _check(load().moe_grouped_gemm_swiglu_gather_save8(_ptr(x), x.shape[0], _ptr(src), int(K), _ptr(w_gate),
                                                       _ptr(w_up), _ptr(offsets), EL, H, F, cap_rows, _ptr(h),
                                                       _ptr(ab8), _ptr(ab8_scale), _handle(stream, dev)))
    return h, ab8, ab8_scale


def moe_grouped_gemm_swiglu_bwd8(dy_perm, w_down, offsets, cap_rows, ab8, ab8_scale, dab=None, h=None,
                                 want_h=True, stream=None):
    """Down dgrad and SwiGLU backward from the 8-bit (a, b) -> (dab, h); want_h=False: h is not recomputed."""
    dev = _device(stream, dy_perm)
    _arg(dy_perm, torch.bfloat16, "dy_perm", dev)
    _arg(w_down, torch.bfloat16, "w_down", dev)
    if w_down.dim() != 3:
        raise MoeError(f"w_down: expected [E, F, H], got {tuple(w_down.shape)}")
    EL, F, H = w_down.shape
    _offsets(offsets, EL, dev)
    _rows(dy_perm, cap_rows, H, "dy_perm")
    _arg(ab8, torch.int8, "ab8", dev)
    _rows(ab8, cap_rows, 2 * F, "ab8")
    _arg(ab8_scale, torch.uint8, "ab8_scale", dev)
    _rows(ab8_scale, cap_rows, 2 * F // 32, "ab8_scale")
    n = max(cap_rows, 0)
    dab = _out(dab, (n, 2 * F), torch.bfloat16, "dab", dev, stream, n)
    h = _out(h, (n, F), torch.bfloat16, "h", dev, stream, n) if want_h else None
    _check(load().moe_grouped_gemm_swiglu_bwd8(_ptr(dy_perm), _ptr(w_down), _ptr(offsets), EL, H, F, cap_rows,
                                               _ptr(ab8), _ptr(ab8_scale), _ptr(dab), _ptr(h), _handle(stream, dev)))
    return dab, h


def pack4_shapes(E, Kd, N):
    """Shapes of (q4, s4) for weights [E, Kd, N]."""
    KT = -(-Kd // 128)
    return (E, N // 16, KT, 64, 16), (E, N // 16, KT, 64)


def _weights4(w, Kd, name, dev, E=None, N=None):
    """Checks a (q4, s4) pair against the contraction length -> (q4, s4, E, N)."""
    q4, s4 = w
    _arg(q4, torch.uint8, name, dev)
    _arg(s4, torch.uint8, name, dev)
    if E is None:
        if q4.dim() != 5:
            raise MoeError(f"{name}: expected 5 dimensions of q4, got {tuple(q4.shape)}")
        E, N = q4.shape[0], q4.shape[1] * 16
    q_shape, s_shape = pack4_shapes(E, Kd, N)
    _shape(q4, q_shape, name)
    _shape(s4, s_shape, name)
    return q4, s4, E, N


def moe_pack4(w, q4=None, s4=None, stream=None):
    """Weights bf16 [E, Kd, N] -> (q4, s4) in 4-bit blocks of 32 along Kd (layout in moe.h)."""
    dev = _device(stream, w)
    _arg(w, torch.bfloat16, "w", dev)
    if w.dim() != 3 or w.shape[1] % 64 or w.shape[2] % 64:
        raise MoeError(f"w: expected [E, Kd, N] with Kd and N multiples of 64, got {tuple(w.shape)}")
    E, Kd, N = w.shape
    q_shape, s_shape = pack4_shapes(E, Kd, N)
    q4 = _out(q4, q_shape, torch.uint8, "q4", dev, stream)
    s4 = _out(s4, s_shape, torch.uint8, "s4", dev, stream)
    _check(load().moe_pack4(_ptr(w), E, Kd, N, _ptr(q4), _ptr(s4), _handle(stream, dev)))
    return q4, s4


def moe_unpack4(q4, s4, Kd, w=None, stream=None):
    """The bf16 weights [E, Kd, N] that (q4, s4) stand for."""
    dev = _device(stream, q4)
    q4, s4, E, N = _weights4((q4, s4), Kd, "w", dev)
    w = _out(w, (E, Kd, N), torch.bfloat16, "w", dev, stream)
    _check(load().moe_unpack4(_ptr(q4), _ptr(s4), E, Kd, N, _ptr(w), _handle(stream, dev)))
    return w


def moe_grouped_gemm4_swiglu(x, src, K, gate, up, offsets, cap_rows, h=None, stream=None):
    """Gate/up product and SwiGLU on 4-bit weights (gate, up: (q4, s4) pairs), row r from x[src[r] // K], or
    from x[r] if src is None (rows already in expert order; K unused)."""
    dev = _device(stream, x)
    _arg(x, torch.bfloat16, "x", dev)
    if x.dim() != 2:
        raise MoeError(f"x: expected [T, H], got {tuple(x.shape)}")
    T, H = x.shape
    gq, gs, EL, F = _weights4(gate, H, "gate", dev)
    uq, us, _, _ = _weights4(up, H, "up", dev, EL, F)
    _offsets(offsets, EL, dev)
    if src is None:
        _rows(x, cap_rows, H, "x")
    else:
        _arg(src, torch.int32, "src", dev)
        if src.numel() < cap_rows:
            raise MoeError(f"src: expected at least {cap_rows} entries, got {src.numel()}")
    n = max(cap_rows, 0)
    h = _out(h, (n, F), torch.bfloat16, "h", dev, stream, n)
    _check(load().moe_grouped_gemm4_swiglu(_ptr(x), T, _ptr(src), int(K or 0), _ptr(gq), _ptr(gs), _ptr(uq),
                                           _ptr(us), _ptr(offsets), EL, H, F, cap_rows, _ptr(h),
                                           _handle(stream, dev)))
    return h


def moe_grouped_gemm4(a, w, offsets, cap_rows, c=None, stream=None):
    """c[r] = a[r] . w_j on 4-bit weights w = (q4, s4); rows in expert order."""
    dev = _device(stream, a)
    _arg(a, torch.bfloat16, "a", dev)
    if a.dim() != 2 or a.shape[0] < cap_rows:
        raise MoeError(f"a: expected at least {cap_rows} rows, got {tuple(a.shape)}")
    Kd = a.shape[1]
    q4, s4, EL, N = _weights4(w, Kd, "w", dev)
    _offsets(offsets, EL, dev)
    n = max(cap_rows, 0)
    c = _out(c, (n, N), torch.bfloat16, "c", dev, stream, n)
    _check(load().moe_grouped_gemm4(_ptr(a), _ptr(q4), _ptr(s4), _ptr(offsets), EL, Kd, N, cap_rows, _ptr(c),
                                    _handle(stream, dev)))
    return c


def moe_gemm4_combine_workspace_size(cap_rows, N) -> int:
    return int(load().moe_gemm4_combine_workspace_size(cap_rows, N))


def moe_grouped_gemm4_combine(a, w, offsets, cap_rows, pos, gates, y=None, out=None, ws=None, stream=None):
    """out[t] = sum_k gates[t,k] * (a[pos[t,k]] . w) on 4-bit weights, the experts' rows kept in fp32 (ws) until
    the one rounding of out; y (optional): those rows in bf16, as moe_grouped_gemm4 gives them."""
    dev = _device(stream, a)
    _arg(a, torch.bfloat16, "a", dev)
    _arg(pos, torch.int32, "pos", dev)
    _arg(gates, torch.float32, "gates", dev)
    if a.dim() != 2 or a.shape[0] < cap_rows:
        raise MoeError(f"a: expected at least {cap_rows} rows, got {tuple(a.shape)}")
    if pos.dim() != 2:
        raise MoeError(f"pos: expected [T, K], got {tuple(pos.shape)}")
    Kd, (T, K) = a.shape[1], pos.shape
    q4, s4, EL, N = _weights4(w, Kd, "w", dev)
    _offsets(offsets, EL, dev)
    _shape(gates, (T, K), "gates")
    if y is not None:
        _arg(y, torch.bfloat16, "y", dev)
        _rows(y, cap_rows, N, "y")
    out = _out(out, (T, N), torch.bfloat16, "out", dev, stream)
    if ws is not None:
        _arg(ws, torch.uint8, "ws", dev)
    need = 4 * max(cap_rows, 0) * N  # as the library's own size, without a call
    if ws is None or ws.numel() < need:
        ws = _empty(max(need, 256), torch.uint8, dev, stream, result=False)
    _check(load().moe_grouped_gemm4_combine(_ptr(a), _ptr(q4), _ptr(s4), _ptr(offsets), EL, Kd, N, cap_rows,
                                            _ptr(pos), _ptr(gates), T, K, _ptr(y), _ptr(out), _ptr(ws), ws.numel(),
                                            _handle(stream, dev)))
    return out


def _ws(ws, need, dev, stream):
    """The caller's workspace, or a new one where there is none or it is too small (None if none is needed)."""
    if ws is not None:
        _arg(ws, torch.uint8, "ws", dev)
    if need == 0 or (ws is not None and ws.numel() >= need):
        return ws, 0 if ws is None else ws.numel()
    return _empty(need, torch.uint8, dev, stream, result=False), need


def _like(t, shape, dtype, name, dev, stream, like):
    """_out for a buffer of a type that the tensor `like` has too, whose allocator is the shorter way to a new one."""
    if t is None and stream is None and like.dtype is dtype:
        return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    return _out(t, shape, dtype, name, dev, stream)


def _rank2(t, name):
    if t.dim() != 2:
        raise MoeError(f"{name}: expected 2 dimensions, got {tuple(t.shape)}")
    return t.shape


def _given(t, shape, dtype, name, dev):
    """An optional input: None, or a tensor of exactly this shape."""
    if t is not None:
        _arg(t, dtype, name, dev)
        _shape(t, shape, name)
    return _ptr(t)


def moe_layer_few_workspace_size(T, K, e_local, H, F) -> int:
    return int(load().moe_layer_few_workspace_size(T, K, e_local, H, F))


def moe_layer_few(logits, x, K, e_begin, w_gate, w_up, w_down, residual=None, topk_idx=None, gates=None, out=None,
                  ws=None, stream=None):
    """The whole layer for at most MOE_FEW_TOKENS tokens on the experts e_begin .. e_begin + e_local - 1 (bf16 weights
    [e_local, H, F] and [e_local, F, H]) -> (out [T, H], topk_idx, gates); residual is added before the one rounding."""
    dev = _device(stream, logits)
    _arg(logits, torch.float32, "logits", dev)
    for t, name in ((x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _arg(t, torch.bfloat16, name, dev)
    T, E = _rank2(logits, "logits")
    if w_gate.dim() != 3:
        raise MoeError(f"w_gate: expected [E, H, F], got {tuple(w_gate.shape)}")
    EL, H, F = w_gate.shape
    _shape(w_up, (EL, H, F), "w_up")
    _shape(w_down, (EL, F, H), "w_down")
    _shape(x, (T, H), "x")
    res = _given(residual, (T, H), torch.bfloat16, "residual", dev)
    K = int(K)
    topk_idx = _out(topk_idx, (T, max(K, 0)), torch.int32, "topk_idx", dev, stream)
    gates = _like(gates, (T, max(K, 0)), torch.float32, "gates", dev, stream, logits)
    out = _like(out, (T, H), torch.bfloat16, "out", dev, stream, x)
    lib = load()
    ws, size = _ws(ws, lib.moe_layer_few_workspace_size(T, K, EL, H, F), dev, stream)
    _check(lib.moe_layer_few(_ptr(logits), _ptr(x), T, E, K, int(e_begin), EL, _ptr(w_gate), _ptr(w_up), _ptr(w_down), H, F,
                             res, _ptr(topk_idx), _ptr(gates), _ptr(out), _ptr(ws), size, _handle(stream, dev)))
    return out, topk_idx, gates


def _stream_type(t, name, dev):
    """The residual stream's type: bf16 (0) or fp32 (1)."""
    f32 = t.dtype is torch.float32
    _arg(t, torch.float32 if f32 else torch.bfloat16, name, dev)
    return int(f32)


def moe_layer_norm(x, weight=None, bias=None, add=None, eps=1e-5, rms=False, sum=None, y=None, mean=None, rstd=None,
                   stream=None):
    """s = x + add and y = bf16((s - mean) * rstd * weight + bias), or of the root mean square with rms -> (s, y, mean,
    rstd); s is x itself without add (and sum), mean is None with rms.  x: bf16 or fp32 [T, H]; sum may be x."""
    dev = _device(stream, x)
    f32 = _stream_type(x, "x", dev)
    T, H = _rank2(x, "x")
    w = _given(weight, (H,), torch.float32, "weight", dev)
    b = _given(bias, (H,), torch.float32, "bias", dev)
    a = _given(add, (T, H), torch.bfloat16, "add", dev)
    if rms and mean is not None:
        raise MoeError("mean: there is none with rms")
    if add is not None or sum is not None:
        sum = _like(sum, (T, H), x.dtype, "sum", dev, stream, x)
    y = _like(y, (T, H), torch.bfloat16, "y", dev, stream, x)
    if not rms:
        mean = _out(mean, (T,), torch.float32, "mean", dev, stream)
    rstd = _out(rstd, (T,), torch.float32, "rstd", dev, stream)
    _check(load().moe_layer_norm(_ptr(x), f32, a, T, H, w, b, eps, int(rms), _ptr(sum), _ptr(y), _ptr(mean),
                                 _ptr(rstd), _handle(stream, dev)))
    return (x if sum is None else sum), y, mean, rstd


def moe_layer_norm_backward_workspace_size(T, H) -> int:
    return int(load().moe_layer_norm_backward_workspace_size(T, H))


def moe_layer_norm_backward(dy, s, weight, mean, rstd, d_sum=None, rms=False, want_dw=True, want_db=None, dx=None,
                            dw=None, db=None, ws=None, stream=None):
    """-> (dx of the type of s, dw, db fp32 [H]; None where not wanted: want_db defaults to there being a mean).
    d_sum, of the type of s, is added to dx, which may be d_sum itself."""
    dev = _device(stream, dy)
    _arg(dy, torch.bfloat16, "dy", dev)
    f32 = _stream_type(s, "s", dev)
    T, H = _rank2(s, "s")
    _shape(dy, (T, H), "dy")
    w = _given(weight, (H,), torch.float32, "weight", dev)
    if rstd is None or (mean is None and not rms):
        raise MoeError("the backward needs the forward's rstd, and its mean unless rms is set")
    m = None if rms else _given(mean, (T,), torch.float32, "mean", dev)
    r = _given(rstd, (T,), torch.float32, "rstd", dev)
    d = _given(d_sum, (T, H), s.dtype, "d_sum", dev)
    want_db = (not rms) if want_db is None else want_db
    if rms and (want_db or db is not None):
        raise MoeError("db: there is no bias with rms")
    dx = _like(dx, (T, H), s.dtype, "dx", dev, stream, s)
    dw = _like(dw, (H,), torch.float32, "dw", dev, stream, rstd) if want_dw or dw is not None else None
    db = _like(db, (H,), torch.float32, "db", dev, stream, rstd) if want_db or db is not None else None
    lib = load()
    need = lib.moe_layer_norm_backward_workspace_size(T, H) if dw is not None or db is not None else 0
    ws, size = _ws(ws, need, dev, stream)
    _check(lib.moe_layer_norm_backward(_ptr(dy), _ptr(s), f32, T, H, w, m, r, int(rms), d, _ptr(dx), _ptr(dw),
                                       _ptr(db), _ptr(ws), size, _handle(stream, dev)))
    return dx, dw, db


def moe_router_bias_backward_workspace_size(T, E) -> int:
    return int(load().moe_router_bias_backward_workspace_size(T, E))


def moe_router_bias_backward(dlogits, dbias=None, ws=None, stream=None):
    """-> dbias fp32 [E], the gradient of moe_router_logits' bias: the column sums of dlogits fp32 [T, E]."""
    dev = _device(stream, dlogits)
    _arg(dlogits, torch.float32, "dlogits", dev)
    T, E = _rank2(dlogits, "dlogits")
    dbias = _like(dbias, (E,), torch.float32, "dbias", dev, stream, dlogits)
    lib = load()
    ws, size = _ws(ws, lib.moe_router_bias_backward_workspace_size(T, E), dev, stream)
    _check(lib.moe_router_bias_backward(_ptr(dlogits), T, E, _ptr(dbias), _ptr(ws), size, _handle(stream, dev)))
    return dbias


def _act(act):
    if act not in ACTS:
        raise MoeError(f"act: expected one of {', '.join(ACTS)}, got {act!r}")
    return ACTS[act]


def moe_linear_workspace_size(T, Kd, N) -> int:
    return int(load().moe_linear_workspace_size(T, Kd, N))


def moe_linear(x, w, bias=None, act="none", residual=None, want_z=False, z=None, y=None, ws=None, stream=None):
    """y = bf16(act(x . w + bias) + residual) -> (y, z), z the bf16 pre-activation if wanted (or its buffer given), else
    None.  x bf16 [T, Kd], w bf16 [Kd, N], bias fp32 [N], act one of ACTS; residual bf16 [T, N] may be y."""
    dev = _device(stream, x)
    _arg(x, torch.bfloat16, "x", dev)
    _arg(w, torch.bfloat16, "w", dev)
    T, Kd = _rank2(x, "x")
    N = _rank2(w, "w")[1]
    _shape(w, (Kd, N), "w")
    b = _given(bias, (N,), torch.float32, "bias", dev)
    res = _given(residual, (T, N), torch.bfloat16, "residual", dev)
    code = _act(act)
    z = _like(z, (T, N), torch.bfloat16, "z", dev, stream, x) if want_z or z is not None else None
    y = _like(y, (T, N), torch.bfloat16, "y", dev, stream, x)
    lib = load()
    ws, size = _ws(ws, lib.moe_linear_workspace_size(T, Kd, N), dev, stream)
    _check(lib.moe_linear(_ptr(x), T, Kd, _ptr(w), N, b, code, res, _ptr(z), _ptr(y), _ptr(ws), size,
                          _handle(stream, dev)))
    return y, z


def moe_linear_backward_workspace_size(T, Kd, N) -> int:
    return int(load().moe_linear_backward_workspace_size(T, Kd, N))


def moe_linear_backward(dy, x, w, act="none", z=None, want_dx=True, want_dw=True, want_db=True, dz=None, dx=None,
                        dw=None, db=None, ws=None, stream=None):
    """-> (dz, dx bf16, dw fp32 [Kd, N], db fp32 [N]; None where not wanted).  dz is dy itself without an activation;
    with one, z is the forward's, and dz may be given (dy itself too)."""
    dev = _device(stream, dy)
    for t, name in ((dy, "dy"), (x, "x"), (w, "w")):
        _arg(t, torch.bfloat16, name, dev)
    T, Kd = _rank2(x, "x")
    N = _rank2(w, "w")[1]
    _shape(w, (Kd, N), "w")
    _shape(dy, (T, N), "dy")
    code = _act(act)
    if code:
        if z is None:
            raise MoeError("z: the backward of an activation needs the forward's")
        zp = _given(z, (T, N), torch.bfloat16, "z", dev)
        dz = _like(dz, (T, N), torch.bfloat16, "dz", dev, stream, dy)
    else:
        if dz is not None and dz is not dy:
            raise MoeError("dz: it is dy itself without an activation")
        zp, dz = None, None
    dx = _like(dx, (T, Kd), torch.bfloat16, "dx", dev, stream, x) if want_dx or dx is not None else None
    dw = _out(dw, (Kd, N), torch.float32, "dw", dev, stream) if want_dw or dw is not None else None
    db = _out(db, (N,), torch.float32, "db", dev, stream) if want_db or db is not None else None
    lib = load()
    need = lib.moe_linear_backward_workspace_size(T, Kd, N) if dw is not None or db is not None else 0
    ws, size = _ws(ws, need, dev, stream)
    _check(lib.moe_linear_backward(_ptr(dy), _ptr(x), T, Kd, _ptr(w), N, code, zp, _ptr(dz), _ptr(dx), _ptr(dw),
                                   _ptr(db), _ptr(ws), size, _handle(stream, dev)))
    return (dy if dz is None else dz), dx, dw, db


def moe_probe_mfma(operands, iters, out=None, stream=None):
    """Measurement aid: back-to-back bf16 MFMAs on register-held operands.
    operands bf16 [blocks*4, 8, 64, 8] (per wave: 4 A then 4 B fragments) -> out fp32 [blocks*4, 64]."""
    _need(operands, torch.bfloat16, "operands")
    if operands.dim() != 4 or tuple(operands.shape[1:]) != (8, 64, 8) or operands.shape[0] % 4:
        raise MoeError(f"operands: expected shape (4*blocks, 8, 64, 8), got {tuple(operands.shape)}")
    waves = operands.shape[0]
    if out is None:
        out = _empty((waves, 64), torch.float32, operands.device, stream)
    _need(out, torch.float32, "out")
    _shape(out, (waves, 64), "out")
    _check(load().moe_probe_mfma(_ptr(operands), waves // 4, iters, _ptr(out), _stream(stream)))
    return out


def moe_probe_mfma16(operands, iters, out=None, stream=None):
    """The probe on 16x16x32 MFMAs: operands bf16 [blocks*4, 16, 64, 8] (per wave: 8 A then 8 B fragments)
    -> out fp32 [blocks*4, 64]."""
    _need(operands, torch.bfloat16, "operands")
    if operands.dim() != 4 or tuple(operands.shape[1:]) != (16, 64, 8) or operands.shape[0] % 4:
        raise MoeError(f"operands: expected shape (4*blocks, 16, 64, 8), got {tuple(operands.shape)}")
    waves = operands.shape[0]
    if out is None:
        out = _empty((waves, 64), torch.float32, operands.device, stream)
    _need(out, torch.float32, "out")
    _shape(out, (waves, 64), "out")
    _check(load().moe_probe_mfma16(_ptr(operands), waves // 4, iters, _ptr(out), _stream(stream)))
    return out


def moe_probe_copy(src, dst, nontemporal=0, blocks=0, stream=None):
    """Measurement aid: a plain streaming copy of src into dst (contiguous device tensors of the same
    byte size, a multiple of 16).  nontemporal: bit 0 loads, bit 1 stores; blocks 0 = 8 per CU."""
    for name, t in (("src", src), ("dst", dst)):
        if not t.is_cuda or not t.is_contiguous():
            raise MoeError(f"{name}: expected a contiguous device tensor")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise MoeError("src and dst differ in byte size")
    _check(load().moe_probe_copy(_ptr(src), _ptr(dst), nbytes, nontemporal, blocks, _stream(stream)))
    return dst
