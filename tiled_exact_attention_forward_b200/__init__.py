"""B200 (sm_100a) tiled exact attention: a thin ctypes binding over libfa_b200.so.

Every step of the computation runs in the CUDA library's kernels; this module
only checks tensor shapes, allocates outputs and workspaces with torch, and
passes raw device pointers and the current CUDA stream to the C ABI declared
in ``include/fa.h``.  There is no CPU fallback: if the library or a CUDA
device is missing, calls raise.

Functions (names follow the C ABI):
    forward(q, k, v, causal=False, window=0, scale=None)        -> (o, lse)
    decode(q, kcache, vcache, seqlens, scale=None)               -> (o, lse)
    decode_paged(q, kpool, vpool, block_table, seqlens)          -> (o, lse)
    backward(q, k, v, o, dout, lse, causal=False, window=0,
             scale=None)                                         -> (dq, dk, dv)
    forward_offset(q, k, v, q_offset, causal=False, window=0)   -> (o, lse)
    merge(o_parts, lse_parts)                                    -> (o, lse)
    norm_rope(q, k, q_weight, k_weight, rope, positions)         -> (q, k) normed and rotated
    norm_rope_backward(q, k, dq_out, dk_out, ...)                -> (dq, dk, dq_weight, dk_weight)
    qk_norm_rope(q, k, q_weight, k_weight, rope, positions)      -> the same (q, k), differentiable
    append_paged(k, v, kpool, vpool, block_table, seqlens)       -> new tokens into a paged cache
    extend_paged(q, kpool, vpool, block_table, seqlens)          -> (o, lse) of new tokens over it
    forward_host(...)  -- forward on pinned host tensors (copies in and out)
    forward_backward_host(...)  -- forward and backward on pinned host tensors
    attention(q, k, v, causal=False, window=0, scale=None)      -> o, differentiable
    device_status()    -- FA_OK or the first recorded device-side timeout

The ring (context-parallel) forward over torch.distributed ranks sits in
``context_parallel``; its compute is ``forward_offset`` and ``merge``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_b200.so")

FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_BF16, FA_FP32, FA_FP16 = 0, 1, 2

EXPORTED_SYMBOLS = (
    "fa_forward",
    "fa_forward_offset",
    "fa_merge",
    "fa_decode_workspace_size",
    "fa_decode",
    "fa_decode_noalloc",
    "fa_decode_paged",
    "fa_backward_workspace_size",
    "fa_backward",
    "fa_norm_rope",
    "fa_norm_rope_backward_workspace_size",
    "fa_norm_rope_backward",
    "fa_append_paged",
    "fa_extend_paged_workspace_size",
    "fa_extend_paged",
    "fa_get_device_status",
    "fa_selftest_wait_timeout",
    "fa_selftest_exp2_poly",
    "fa_status_string",
    "fa_version",
)


class FAError(RuntimeError):
    """A non-FA_OK status from the C ABI."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib().fa_status_string(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg}")


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m tiled_exact_attention_forward_b200.build`"
        )
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_forward.argtypes = [P, P, P, P, P, I, I, I, I, F, I, I, I, P]
    lib.fa_forward.restype = I
    lib.fa_forward_offset.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, I, I, P]
    lib.fa_forward_offset.restype = I
    lib.fa_merge.argtypes = [P, P, I, P, P, I, I, I, I, I, P]
    lib.fa_merge.restype = I
    lib.fa_decode_workspace_size.argtypes = [I, I, I, I]
    lib.fa_decode_workspace_size.restype = Z
    lib.fa_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, F, I, P, Z, P]
    lib.fa_decode.restype = I
    lib.fa_decode_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, F, I, P]
    lib.fa_decode_noalloc.restype = I
    lib.fa_decode_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
    lib.fa_decode_paged.restype = I
    lib.fa_backward_workspace_size.argtypes = [I, I, I, I]
    lib.fa_backward_workspace_size.restype = Z
    lib.fa_backward.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, I, I, P, Z, P]
    lib.fa_backward.restype = I
    L = ctypes.c_longlong
    lib.fa_norm_rope.argtypes = [P] * 9 + [L] + [I] * 7 + [F, I, I, I, P]
    lib.fa_norm_rope.restype = I
    lib.fa_norm_rope_backward_workspace_size.argtypes = [I]
    lib.fa_norm_rope_backward_workspace_size.restype = Z
    lib.fa_norm_rope_backward.argtypes = [P] * 13 + [L] + [I] * 7 + [F, I, I, I, P, Z, P]
    lib.fa_norm_rope_backward.restype = I
    lib.fa_append_paged.argtypes = [P] * 9 + [L] * 3 + [P] * 3 + [I] * 10 + [F, I, I, I, P]
    lib.fa_append_paged.restype = I
    lib.fa_extend_paged_workspace_size.argtypes = [I, I, I, I]
    lib.fa_extend_paged_workspace_size.restype = Z
    lib.fa_extend_paged.argtypes = [P] * 8 + [L] + [I] * 8 + [F, I, I, I, P, Z, P]
    lib.fa_extend_paged.restype = I
    lib.fa_selftest_wait_timeout.argtypes = [ctypes.c_longlong, P]
    lib.fa_selftest_wait_timeout.restype = I
    lib.fa_selftest_exp2_poly.argtypes = [P, P, ctypes.c_longlong, P]
    lib.fa_selftest_exp2_poly.restype = I
    lib.fa_get_device_status.argtypes = [P]
    lib.fa_get_device_status.restype = I
    lib.fa_status_string.argtypes = [I]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = I
    _LIB = lib
    return lib


def library() -> ctypes.CDLL:
    """The loaded C library (raises ImportError if it has not been built)."""
    return _lib()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, where: str):
    if status != FA_OK:
        raise FAError(status, where)


_DTYPE_CODES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16, torch.float32: FA_FP32}


def _dtype_code(dt: torch.dtype) -> int:
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}: use torch.bfloat16, torch.float16 or torch.float32")
    return code


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device (there is no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if t.device != ts[0].device:
            raise ValueError("tensors must all be on the same CUDA device")


def _scale_arg(scale) -> float:
    return 0.0 if scale is None else float(scale)


def forward(q, k, v, causal: bool = False, window: int = 0, scale=None, out=None, lse=None):
    """O = softmax(q k^T * scale + mask) v and the float32 row logsumexp.

    q, k, v: [B, H, N, d] contiguous CUDA tensors (bf16 or fp16 with d = 128, or
    fp32 with d in {64, 128}).  Returns (o, lse) with o like q and lse [B, H, N].
    """
    _need_cuda(q, k, v)
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share shape and dtype")
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = _lib().fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                           _scale_arg(scale), int(bool(causal)), int(window),
                           _dtype_code(q.dtype), _stream(q.device))
    _check(st, "fa_forward")
    return o, lse


def forward_offset(q, k, v, q_offset: int, causal: bool = False, window: int = 0, scale=None,
                   out=None, lse=None):
    """One key shard's partial forward (context parallelism).

    q: [B, H, Nq, d]; k, v: [B, H, Nk, d] (bf16 or fp16, d = 128), contiguous CUDA
    tensors.  Query row i sits at position i + q_offset of the key sequence; the
    causal and window masks are taken at those positions.  Returns (o, lse): the
    softmax over these keys only, o like q, lse [B, H, Nq] (-inf, with o = 0, for
    a row that sees none of the keys).
    """
    _need_cuda(q, k, v)
    B, H, Nq, d = q.shape
    if k.dim() != 4 or k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Nk, d] with q's B, H and d")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype")
    Nk = k.shape[2]
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    st = _lib().fa_forward_offset(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk,
                                  int(q_offset), d, _scale_arg(scale), int(bool(causal)), int(window),
                                  _dtype_code(q.dtype), _stream(q.device))
    _check(st, "fa_forward_offset")
    return o, lse


def merge(o_parts, lse_parts, out=None, lse=None):
    """Combine S partial results over disjoint key sets into the full attention.

    o_parts: [S, B, H, N, d] (bf16, fp16 or float32, d in {64, 128}); lse_parts:
    [S, B, H, N] float32 (-inf marks a part that saw no key for that row).
    Returns (o [B, H, N, d] in the parts' dtype, lse [B, H, N]).
    """
    _need_cuda(o_parts, lse_parts)
    S, B, H, N, d = o_parts.shape
    if lse_parts.shape != (S, B, H, N) or lse_parts.dtype != torch.float32:
        raise ValueError("lse_parts must be float32 [S, B, H, N] matching o_parts")
    o = torch.empty(o_parts.shape[1:], dtype=o_parts.dtype, device=o_parts.device) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=o_parts.device)
    st = _lib().fa_merge(_ptr(o_parts), _ptr(lse_parts), S, _ptr(o), _ptr(lse), B, H, N, d,
                         _dtype_code(o_parts.dtype), _stream(o_parts.device))
    _check(st, "fa_merge")
    return o, lse


_HOST_STREAMS = {}


def _host_streams(dev):
    """Three side streams per device (copy in, compute, copy out), made once."""
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    if key not in _HOST_STREAMS:
        _HOST_STREAMS[key] = tuple(torch.cuda.Stream(device=dev) for _ in range(3))
    return _HOST_STREAMS[key]


def _host_pipelined(dev, host_ins, out_specs, chunks, compute):
    """Runs `compute` over head groups with the copies pipelined around it.

    host_ins: host tensors whose first dimension is the B * H heads; out_specs:
    (trailing shape, dtype) of each output, also head-major.  For each group of
    heads [a, b): the inputs are copied in on one stream, compute(a, b, dev_ins,
    dev_outs) runs on a second, the outputs are copied back on a third, so the
    copy-in of one group overlaps the kernels of the previous group and the
    copy-out of the one before (PCIe moves both directions at once).  The
    copy-in stream first waits for the work already queued on the current
    stream; the call returns once the results are in (pinned) host memory.
    """
    BH = host_ins[0].shape[0]
    chunks = max(1, min(int(chunks), BH))
    dev_ins = [torch.empty(t.shape, dtype=t.dtype, device=dev) for t in host_ins]
    dev_outs = [torch.empty((BH, *tail), dtype=dt, device=dev) for tail, dt in out_specs]
    host_outs = [torch.empty((BH, *tail), dtype=dt, pin_memory=True) for tail, dt in out_specs]
    s_in, s_run, s_out = _host_streams(dev)
    cur = torch.cuda.current_stream(dev)
    s_in.wait_stream(cur)
    bounds = [(g * BH) // chunks for g in range(chunks + 1)]
    for g in range(chunks):
        a, b = bounds[g], bounds[g + 1]
        with torch.cuda.stream(s_in):
            for dst, src in zip(dev_ins, host_ins):
                dst[a:b].copy_(src[a:b], non_blocking=True)
        s_run.wait_stream(s_in)
        with torch.cuda.stream(s_run):
            compute(a, b, dev_ins, dev_outs)
        s_out.wait_stream(s_run)
        with torch.cuda.stream(s_out):
            for dst, src in zip(host_outs, dev_outs):
                dst[a:b].copy_(src[a:b], non_blocking=True)
    cur.wait_stream(s_out)
    s_out.synchronize()
    return host_outs, max(bounds[g + 1] - bounds[g] for g in range(chunks))


def _check_host(*ts):
    for t in ts:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host-buffer calls take contiguous host tensors")
    if any(t.shape != ts[0].shape or t.dtype != ts[0].dtype for t in ts):
        raise ValueError("q, k, v (and dout) must share shape and dtype")


def forward_host(q, k, v, causal: bool = False, window: int = 0, scale=None, device="cuda", chunks: int = 4):
    """The forward for host tensors: copy in, run, copy out; returns pinned host (o, lse).

    q, k, v: contiguous [B, H, N, d] host tensors (pinned memory makes the copies
    asynchronous).  Every (batch, head) is independent, so the heads go through
    in `chunks` groups with copies and kernels overlapped (see _host_pipelined).
    """
    _check_host(q, k, v)
    dev = torch.device(device)
    B, H, N, d = q.shape

    def run(a, b, ins, outs):
        qd, kd, vd = (t[a:b].unsqueeze(0) for t in ins)
        forward(qd, kd, vd, causal, window, scale, out=outs[0][a:b].unsqueeze(0), lse=outs[1][a:b].unsqueeze(0))

    (o, lse), _ = _host_pipelined(dev, [t.reshape(B * H, N, d) for t in (q, k, v)],
                                  [((N, d), q.dtype), ((N,), torch.float32)], chunks, run)
    return o.view(B, H, N, d), lse.view(B, H, N)


def forward_backward_host(q, k, v, dout, causal: bool = False, window: int = 0, scale=None, device="cuda",
                          chunks: int = 8):
    """Forward and backward for host tensors; returns pinned host (o, lse, dq, dk, dv).

    The heads go through in `chunks` groups with copies and kernels overlapped
    (see _host_pipelined); the backward's workspace is sized for the largest
    group and reused, the groups' kernels running in order on one stream.
    """
    _check_host(q, k, v, dout)
    dev = torch.device(device)
    B, H, N, d = q.shape
    chunks = max(1, min(int(chunks), B * H))
    largest = -(-(B * H) // chunks)
    ws = torch.empty(max(backward_workspace_size(1, largest, N, d), 256), dtype=torch.uint8, device=dev)

    def run(a, b, ins, outs):
        qd, kd, vd, gd = (t[a:b].unsqueeze(0) for t in ins)
        od, ld, dqd, dkd, dvd = (t[a:b].unsqueeze(0) for t in outs)
        forward(qd, kd, vd, causal, window, scale, out=od, lse=ld)
        backward(qd, kd, vd, od, gd, ld, causal, window, scale, workspace=ws, dq=dqd, dk=dkd, dv=dvd)

    specs = [((N, d), q.dtype), ((N,), torch.float32)] + [((N, d), q.dtype)] * 3
    outs, _ = _host_pipelined(dev, [t.reshape(B * H, N, d) for t in (q, k, v, dout)], specs, chunks, run)
    o, lse, dq, dk, dv = outs
    return o.view(B, H, N, d), lse.view(B, H, N), dq.view(B, H, N, d), dk.view(B, H, N, d), dv.view(B, H, N, d)


def decode_workspace_size(B, H, cap, d) -> int:
    return int(_lib().fa_decode_workspace_size(B, H, cap, d))


def decode(q, kcache, vcache, seqlens, scale=None, workspace=None, out=None, lse=None):
    """Single-token decode: q [B, H, d] against kcache/vcache [B, H, cap, d].

    seqlens: int32 [B] CUDA tensor; query (b, h) attends to cache rows
    j < seqlens[b].  Returns (o [B, H, d] bf16, lse [B, H] float32).
    """
    _need_cuda(q, kcache, vcache, seqlens)
    B, H, d = q.shape
    cap = kcache.shape[2]
    if kcache.shape != (B, H, cap, d) or vcache.shape != kcache.shape:
        raise ValueError("kcache/vcache must be [B, H, cap, d] matching q")
    if kcache.dtype != q.dtype or vcache.dtype != q.dtype:
        raise ValueError("kcache/vcache must have q's dtype")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    need = decode_workspace_size(B, H, cap, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = _lib().fa_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(o), _ptr(lse),
                          B, H, cap, d, _scale_arg(scale), _dtype_code(q.dtype),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _stream(q.device))
    _check(st, "fa_decode")
    return o, lse


def decode_paged(q, kpool, vpool, block_table, seqlens, scale=None, workspace=None, out=None, lse=None):
    """Single-token decode against a paged cache.

    q [B, H, d]; kpool/vpool [num_blocks, H, block_size, d] (block_size a power
    of two); block_table int32 [B, max_blocks] maps sequence b's logical block t
    (keys [t * block_size, (t + 1) * block_size)) to a pool block; seqlens int32
    [B].  Returns (o [B, H, d] bf16, lse [B, H] float32).  An out-of-range block
    id of a used block is skipped and reported by device_status().
    """
    _need_cuda(q, kpool, vpool, block_table, seqlens)
    B, H, d = q.shape
    num_blocks, _, bs, _ = kpool.shape
    if kpool.shape != (num_blocks, H, bs, d) or vpool.shape != kpool.shape:
        raise ValueError("kpool/vpool must be [num_blocks, H, block_size, d] matching q")
    if kpool.dtype != q.dtype or vpool.dtype != q.dtype:
        raise ValueError("kpool/vpool must have q's dtype")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be an int32 tensor of shape [B, max_blocks]")
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be an int32 tensor of shape [B]")
    max_blocks = block_table.shape[1]
    need = decode_workspace_size(B, H, max_blocks * bs, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = _lib().fa_decode_paged(_ptr(q), _ptr(kpool), _ptr(vpool), _ptr(block_table), _ptr(seqlens),
                                _ptr(o), _ptr(lse), B, H, num_blocks, bs, max_blocks, d, _scale_arg(scale),
                                _dtype_code(q.dtype), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(q.device))
    _check(st, "fa_decode_paged")
    return o, lse


def backward_workspace_size(B, H, N, d) -> int:
    return int(_lib().fa_backward_workspace_size(B, H, N, d))


def backward(q, k, v, o, dout, lse, causal: bool = False, window: int = 0, scale=None,
             workspace=None, dq=None, dk=None, dv=None):
    """Gradients (dq, dk, dv) of the forward, recomputing P from lse."""
    _need_cuda(q, k, v, o, dout, lse)
    B, H, N, d = q.shape
    for t in (k, v, o, dout):
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError("q, k, v, o, dout must share shape and dtype")
    if lse.shape != (B, H, N) or lse.dtype != torch.float32:
        raise ValueError("lse must be float32 [B, H, N]")
    need = backward_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    st = _lib().fa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                            _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, _scale_arg(scale),
                            int(bool(causal)), int(window), _dtype_code(q.dtype),
                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                            _stream(q.device))
    _check(st, "fa_backward")
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    """forward keeps (q, k, v, o, lse); backward recomputes P from lse in the library."""

    @staticmethod
    def forward(ctx, q, k, v, causal, window, scale):
        o, lse = forward(q, k, v, causal, window, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.mask = (causal, window, scale)
        return o

    @staticmethod
    def backward(ctx, grad_o):
        q, k, v, o, lse = ctx.saved_tensors
        causal, window, scale = ctx.mask
        dq, dk, dv = backward(q, k, v, o, grad_o.contiguous(), lse, causal, window, scale)
        return dq, dk, dv, None, None, None


def attention(q, k, v, causal: bool = False, window: int = 0, scale=None):
    """Differentiable attention: o = softmax(q k^T * scale + mask) v with autograd.

    The forward runs the library's forward and saves the row logsumexp; the
    backward runs the library's backward, which recomputes P from it (bf16,
    d = 128 for the backward).  Gradients stay on the device.
    """
    return _Attention.apply(q, k, v, bool(causal), int(window), scale)


# The calls below are made once or more per layer and token, so their host time counts:
# checks are plain comparisons, pointers and strides go to the C ABI as integers and
# packed bytes (about 25 microseconds a call became 12).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_pack12 = struct.Struct("12q").pack
_pack18 = struct.Struct("18q").pack


def _on(first, *others):
    """The CUDA device index of `first`; every other given tensor must sit there (None: skipped)."""
    i = first.get_device()
    if i < 0:
        raise ValueError("tensors must be on a CUDA device (there is no CPU path)")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError("tensors must all be on the same CUDA device")
    return i


def _launch(fn, name, device, *args):
    """fn(*args, stream) with `device` current and its current stream; raises on a non-FA_OK status."""
    if _current_device() == device:
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st != FA_OK:
        raise FAError(st, name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _need_int32(name, t, shape):
    if t.shape != shape or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)}")


def _strides(t, packed):
    """(batch, head, row) strides of a [B, H, N, d] or packed [T, H, d] tensor with contiguous rows."""
    st = t.stride()
    if st[-1] != 1:
        raise ValueError("the rows (last dimension) of q, k, their outputs and gradients must be contiguous")
    return (0, st[1], st[0]) if packed else st[:3]


def _qk_sizes(q, k):
    """(B, Hq, Hk, N, d, packed) of queries and keys, [B, H, N, d] or packed [T, H, d]."""
    shape = q.shape
    packed = len(shape) == 3
    if packed:
        N, Hq, d = shape
        B = 1
    elif len(shape) == 4:
        B, Hq, N, d = shape
    else:
        raise ValueError("q must be [B, H, N, d] or packed [T, H, d]")
    if k is None:
        return B, Hq, 0, N, d, packed
    Hk = k.shape[1]
    if k.shape != ((N, Hk, d) if packed else (B, Hk, N, d)) or k.dtype != q.dtype:
        raise ValueError("q and k must share dtype and every size but the heads")
    return B, Hq, Hk, N, d, packed


def _grad_like(t):
    """An uninitialised gradient laid out as t where t is dense, contiguous where not (expanded views)."""
    g = torch.empty_like(t)
    return g if g.stride(-1) == 1 else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _readable(g):
    """g, or a copy where the kernels cannot read it in place (its layout is what autograd made of it)."""
    e = g.element_size()
    if g.stride(-1) == 1 and g.data_ptr() % 16 == 0:
        if all(n < 2 or st * e % 16 == 0 for n, st in zip(g.shape[:-1], g.stride())):
            return g
    return g.clone(memory_format=torch.contiguous_format)


def _rotation_args(dtype, q_weight, k_weight, rope, eps, d):
    """(rot, max_pos, eps for the C ABI, weight dtype code) of a norm and rotation."""
    rot = max_pos = 0
    if rope is not None:
        shape = rope.shape
        if len(shape) != 2 or rope.dtype != torch.float32 or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 tensor [positions, rot]: rot/2 cosines, rot/2 sines")
        max_pos, rot = shape
        if rot == 0 or rot % 16 or rot > d:
            raise ValueError("rope's second dimension must be a multiple of 16 up to the head dimension")
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights need eps: without it there is no norm")
        return rot, max_pos, -1.0, _dtype_code(dtype)
    if not eps >= 0:
        raise ValueError("eps must be >= 0 (None: no norm)")
    wdt = None
    for w in (q_weight, k_weight):
        if w is not None:
            t = w.dtype
            if w.shape != (d,) or not w.is_contiguous():
                raise ValueError("weights must be contiguous tensors of the head dimension")
            if (t != dtype and t != torch.float32) or (wdt is not None and t != wdt):
                raise ValueError("weights must share one dtype: the tensors' or float32")
            wdt = t
    return rot, max_pos, float(eps), _dtype_code(dtype if wdt is None else wdt)


def _position_stride(positions, B, N):
    if positions is None:
        return 0
    if positions.dtype != torch.int32 or positions.shape not in ((N,), (B, N)) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 tensor [N] or [B, N] (packed: [T])")
    return N if positions.dim() == 2 else 0


def _out_like(x, out):
    """An output of x's sizes: the given one, checked, or a new contiguous one."""
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("an output must have its input's shape and dtype")
    return out


_NO_STRIDES = (0, 0, 0)


def norm_rope(q, k=None, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6,
              interleaved: bool = False, q_out=None, k_out=None):
    """Per-head RMS norm and position rotation of queries and keys in one launch.

    q, k: [B, H, N, d] (or packed [T, H, d]) CUDA tensors, d in {64, 128}, bf16,
    fp16 or float32, rows contiguous, other strides free (multiples of 16 bytes):
    a transposed view of a projection's [B, N, H, d] output is read where it lies.
    H may differ between q and k; k may be None.
    y = x / sqrt(mean(x^2) + eps) * weight per row (weight [d], None for ones;
    eps=None leaves the norm out), then the first rot elements turned by the angles of
    the row's position.  rope: float32 [positions, rot], rot/2 cosines then rot/2
    sines per position, rot a multiple of 16 (None: no rotation); pairs are
    (i, i + rot/2), or (2i, 2i + 1) with interleaved.  positions: int32 [N] or [B, N]
    (packed: [T]); None: 0 .. N-1.  A position outside the table gives NaN and is
    reported by device_status().
    Returns (q_out, k_out), contiguous [B, H, N, d] (or [T, H, d]), as the attention
    calls take them; without k, q_out alone.  q_out, k_out may be given (at any
    strides, the inputs themselves among them).
    """
    device = _on(q, k, q_weight, k_weight, rope, positions, q_out, k_out)
    B, Hq, Hk, N, d, packed = _qk_sizes(q, k)
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("k_weight and k_out need k")
    rot, max_pos, e, wcode = _rotation_args(q.dtype, q_weight, k_weight, rope, eps, d)
    pos_stride = _position_stride(positions, B, N)
    q_out = _out_like(q, q_out)
    ks = kos = _NO_STRIDES
    if k is not None:
        k_out = _out_like(k, k_out)
        ks, kos = _strides(k, packed), _strides(k_out, packed)
    strides = _pack12(*_strides(q, packed), *ks, *_strides(q_out, packed), *kos)
    _launch(_lib().fa_norm_rope, "fa_norm_rope", device, q.data_ptr(), _addr(k), q_out.data_ptr(), _addr(k_out),
            strides, _addr(q_weight), _addr(k_weight), _addr(rope), _addr(positions), pos_stride, B, Hq, Hk, N, d, rot, max_pos, e, int(bool(interleaved)),
            _dtype_code(q.dtype), wcode)
    return (q_out, k_out) if k is not None else q_out


@functools.lru_cache(maxsize=None)
def norm_rope_backward_workspace_size(d) -> int:
    return int(_lib().fa_norm_rope_backward_workspace_size(d))


def norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6,
                       interleaved: bool = False, workspace=None):
    """Gradients of norm_rope: (dq, dk, dq_weight, dk_weight).

    q, k: the forward's inputs; dq_out, dk_out: the gradients of its outputs, of the
    same sizes, rows contiguous.  k and dk_out may be None together (dk is then
    None).  dq and dk are laid out as q and k are (dense in their strides' order).
    A weight that is None has no gradient (None); weight gradients are summed in
    float32 in a fixed order and come in the weights' dtype.
    """
    device = _on(q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, workspace)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    B, Hq, Hk, N, d, packed = _qk_sizes(q, k)
    if dq_out.shape != q.shape or dq_out.dtype != q.dtype:
        raise ValueError("dq_out must have q's shape and dtype")
    dq, dk = _grad_like(q), None
    ks = kgs = dks = _NO_STRIDES
    if k is not None:
        if dk_out.shape != k.shape or dk_out.dtype != k.dtype:
            raise ValueError("dk_out must have k's shape and dtype")
        dk = _grad_like(k)
        ks, kgs, dks = _strides(k, packed), _strides(dk_out, packed), _strides(dk, packed)
    elif k_weight is not None:
        raise ValueError("k_weight needs k")
    rot, max_pos, e, wcode = _rotation_args(q.dtype, q_weight, k_weight, rope, eps, d)
    pos_stride = _position_stride(positions, B, N)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    strides = _pack18(*_strides(q, packed), *ks, *_strides(dq_out, packed), *kgs, *_strides(dq, packed), *dks)
    ws_bytes = 0
    if dqw is not None or dkw is not None:
        if workspace is None:
            workspace = q.new_empty((norm_rope_backward_workspace_size(d),), dtype=torch.uint8)
        ws_bytes = workspace.numel() * workspace.element_size()
    _launch(_lib().fa_norm_rope_backward, "fa_norm_rope_backward", device, q.data_ptr(), _addr(k), dq_out.data_ptr(),
            _addr(dk_out), dq.data_ptr(), _addr(dk), strides, _addr(q_weight), _addr(k_weight), _addr(dqw), _addr(dkw),
            _addr(rope), _addr(positions), pos_stride, B, Hq, Hk,
            N, d, rot, max_pos, e, int(bool(interleaved)), _dtype_code(q.dtype), wcode, _addr(workspace), ws_bytes)
    return dq, dk, dqw, dkw


class _QKNormRope(torch.autograd.Function):
    """Saves the inputs; the backward recomputes the rows' norms from them."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, rope, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, rope, positions)
        ctx.how = (eps, interleaved)
        return norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk=None):
        q, k, q_weight, k_weight, rope, positions = ctx.saved_tensors
        dq, dk, dqw, dkw = norm_rope_backward(q, k, _readable(gq), None if gk is None else _readable(gk), q_weight,
                                              k_weight, rope, positions, *ctx.how)
        return dq, dk, dqw, dkw, None, None, None, None


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, rope=None, positions=None, eps=1e-6,
                 interleaved: bool = False):
    """norm_rope with autograd: gradients for q, k and the weights (rope and positions have none;
    no second derivatives).

    The step before ``attention``: q, k = qk_norm_rope(q, k, ...); o = attention(q, k, v, causal=True).
    To capture forward and backward into a CUDA graph, drop every eager autograd graph of the
    same leaves first, as torch's graph capture asks of any differentiable operation.
    """
    return _QKNormRope.apply(q, k, q_weight, k_weight, rope, positions, eps, bool(interleaved))


def _token_stride(name, t, T, H, d, dtype):
    """The token stride of a packed [T, H, d] tensor whose heads are contiguous."""
    if t.shape != (T, H, d) or t.dtype != dtype:
        raise ValueError(f"{name} must be packed [{T}, {H}, {d}] with the pools' dtype")
    st = t.stride()
    if st[2] != 1 or (st[1] != d and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return st[0]


def _paged_sizes(kpool, vpool, block_table, seqlens, cu_tokens, T):
    """(num_blocks, Hkv, block_size, d, B, max_blocks) of a paged cache, its tensors checked."""
    shape = kpool.shape
    if len(shape) != 4 or vpool.shape != shape or vpool.dtype != kpool.dtype:
        raise ValueError("kpool and vpool must be [num_blocks, Hkv, block_size, d] and share dtype")
    if not (kpool.is_contiguous() and vpool.is_contiguous()):
        raise ValueError("kpool and vpool must be contiguous")
    if block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor of shape [B, max_blocks]")
    B, max_blocks = block_table.shape
    _need_int32("block_table", block_table, (B, max_blocks))
    _need_int32("seqlens", seqlens, (B,))
    if cu_tokens is not None:
        _need_int32("cu_tokens", cu_tokens, (B + 1,))
    elif T != B:
        raise ValueError("without cu_tokens there is one token for each sequence")
    return (*shape, B, max_blocks)


def append_paged(k, v, kpool, vpool, block_table, seqlens, cu_tokens=None, rope=None, q=None, q_weight=None,
                 k_weight=None, eps=None, interleaved: bool = False, q_out=None):
    """New tokens' keys and values into a paged cache, in place, the keys rotated on the way.

    k, v: packed [T, Hkv, d] CUDA tensors (bf16 or fp16, d = 128), tokens at any stride
    (views of a fused projection).  kpool, vpool, block_table as decode_paged takes
    them.  cu_tokens: int32 [B + 1], sequence b's tokens are cu_tokens[b] ..
    cu_tokens[b + 1] - 1 (None: one token each, T = B).  seqlens: int32 [B], the
    lengths WITH the new tokens: the tokens take the last positions, and the same
    array serves extend_paged and decode_paged.
    Keys are normed (eps given, weight k_weight or ones) and turned by rope as in
    norm_rope; values are copied.  q, packed [T, Hq, d], is normed with q_weight and
    turned in the same launch: returned contiguous (None without q, q_weight then unused).
    A token without a place (position outside the cache or the table, block id outside
    the pool) is not written and reported by device_status().
    """
    device = _on(k, v, kpool, vpool, block_table, seqlens, cu_tokens, rope, q, q_weight, k_weight, q_out)
    T = k.shape[0]
    dtype = kpool.dtype
    num_blocks, Hkv, bs, d, B, max_blocks = _paged_sizes(kpool, vpool, block_table, seqlens, cu_tokens, T)
    k_stride, v_stride = _token_stride("k", k, T, Hkv, d, dtype), _token_stride("v", v, T, Hkv, d, dtype)
    rot, max_pos, e, wcode = _rotation_args(dtype, q_weight, k_weight, rope, eps, d)
    Hq = q_stride = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be packed [T, Hq, d]")
        Hq = q.shape[1]
        q_stride = _token_stride("q", q, T, Hq, d, dtype)
        q_out = _out_like(q, q_out)
        if not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _launch(_lib().fa_append_paged, "fa_append_paged", device, k.data_ptr(), v.data_ptr(), _addr(q), _addr(q_out),
            kpool.data_ptr(), vpool.data_ptr(), block_table.data_ptr(), _addr(cu_tokens), seqlens.data_ptr(), q_stride,
            k_stride, v_stride, _addr(q_weight), _addr(k_weight), _addr(rope), T, B, Hq, Hkv, num_blocks, bs, max_blocks,
            d, rot, max_pos, e, int(bool(interleaved)), _dtype_code(dtype), wcode)
    return q_out


@functools.lru_cache(maxsize=4096)
def extend_paged_workspace_size(T, Hq, Hkv, d) -> int:
    return int(_lib().fa_extend_paged_workspace_size(T, Hq, Hkv, d))


def extend_paged(q, kpool, vpool, block_table, seqlens, cu_tokens=None, causal: bool = True, window: int = 0, scale=None,
                 workspace=None, out=None, lse=None):
    """Attention of packed new tokens over a paged cache that holds them already.

    q: packed [T, Hq, d] CUDA tensor (bf16 or fp16, d = 128), tokens at any stride;
    pools, block_table, seqlens and cu_tokens as append_paged takes them, Hq a
    multiple of the pools' heads (query head h reads key head h * Hkv // Hq).  Token i
    of the m new ones of a sequence of length n sits at position n - m + i and sees
    the keys up to itself (causal), the last `window` of them with window > 0.
    Returns (o [T, Hq, d], lse [T, Hq] float32); o = 0 and lse = -inf for a token that
    sees no key; tokens outside every sequence keep what out and lse held.  Calls that
    may overlap need workspaces of their own (the default makes one).  An out-of-range
    block id of a used block is skipped and reported by device_status().
    """
    device = _on(q, kpool, vpool, block_table, seqlens, cu_tokens, workspace, out, lse)
    if q.dim() != 3:
        raise ValueError("q must be packed [T, Hq, d]")
    T, Hq = q.shape[:2]
    dtype = kpool.dtype
    num_blocks, Hkv, bs, d, B, max_blocks = _paged_sizes(kpool, vpool, block_table, seqlens, cu_tokens, T)
    q_stride = _token_stride("q", q, T, Hq, d, dtype)
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the pools' heads")
    out = _out_like(q, out)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if lse is None:
        lse = q.new_empty((T, Hq), dtype=torch.float32)
    elif lse.shape != (T, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [T, Hq]")
    if workspace is None:
        workspace = q.new_empty(max(extend_paged_workspace_size(T, Hq, Hkv, d), 256), dtype=torch.uint8)
    _launch(_lib().fa_extend_paged, "fa_extend_paged", device, q.data_ptr(), kpool.data_ptr(), vpool.data_ptr(),
            block_table.data_ptr(), _addr(cu_tokens), seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(), q_stride, T, B,
            Hq, Hkv, num_blocks, bs, max_blocks, d, _scale_arg(scale), int(bool(causal)), int(window),
            _dtype_code(dtype), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


def selftest_wait_timeout(limit_cycles: int = 20_000_000, device=None) -> int:
    """Run the failure-path self-test kernel (a bounded wait that must expire)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    return int(_lib().fa_selftest_wait_timeout(int(limit_cycles), _stream(dev)))


def device_status(device=None) -> int:
    """Synchronise the current stream and return the library's device status."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    return int(_lib().fa_get_device_status(_stream(dev)))
