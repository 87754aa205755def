"""ctypes binding of the operators beside the quantized product
(include/qmv_ops.h): the adapted projection, the mixture-of-experts layer and
the verification of drafted tokens.

Argument checks and marshalling only: every step runs in the HIP kernels of
lib/libqmv.so, and there is no fallback path.  Outputs and scratch memory are
allocated on the stream that the call runs on.
"""
from __future__ import annotations

import ctypes

from . import qmv
from .qmv import DT_BF16, DT_F16, DT_F32, QmvError

_lib = None
_DT = None          # torch dtype -> qmv_dtype


def _load():
    global _lib, _DT
    if _lib is None:
        import torch
        L = qmv.lib()
        P, I, Q = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        for name, args in (("qmv_affine_lora", [P] * 10 + [Q] + [I] * 11 + [P]),):
            f = getattr(L, name)
            f.argtypes, f.restype = args, I
        for name, n in (("qmv_affine_lora_workspace", 3),):
            f = getattr(L, name)
            f.argtypes, f.restype = [I] * n, Q
        _DT = {torch.float32: DT_F32, torch.float16: DT_F16, torch.bfloat16: DT_BF16}
        _lib = L
    return _lib


class _On:
    """The device and stream a call runs on.  Entered around the allocation of
    its outputs and scratch memory and its launches; where the stream is not the
    current one of the inputs' device, the inputs are recorded on it, so that their
    memory is not handed out again before the call has read it."""

    def __init__(self, dev, stream, inputs):
        import torch
        self.stream = torch.cuda.current_stream(dev) if stream is None else stream
        self.ctx = None
        if torch.cuda.current_device() != dev.index:
            self.ctx = torch.cuda.device(dev)
        if stream is not None and stream != torch.cuda.current_stream(dev):
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the inputs on {dev}")
            self.ctx = torch.cuda.stream(stream)
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _shape(t, name, *shape):
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _dtype(t, name, *allowed):
    if t.dtype not in allowed:
        raise TypeError(f"{name} must be " + " or ".join(str(d).replace("torch.", "") for d in allowed)
                        + f", got {str(t.dtype).replace('torch.', '')}")


def _matrix(w, s, b, lead, K, bits, gs, name):
    """A quantized matrix: packed codes, scales and biases of shape [*lead][...]."""
    import torch
    if bits not in (2, 4):
        raise ValueError(f"bits must be 2 or 4, got {bits}")
    if gs not in (64, 128):
        raise ValueError(f"group_size must be 64 or 128, got {gs}")
    if K < gs or K % gs != 0:
        raise ValueError(f"{name}: {K} columns are not a multiple of group_size = {gs}")
    _dtype(w, name, torch.int32, torch.uint32)
    _dtype(s, f"{name} scales", torch.bfloat16, torch.float16)
    if b.dtype != s.dtype:
        raise TypeError(f"{name}: scales and biases must share a dtype")
    _shape(w, name, *lead, K * bits // 32)
    _shape(s, f"{name} scales", *lead, K // gs)
    _shape(b, f"{name} biases", *lead, K // gs)


def _out(out, out_dtype, shape, dev, torch):
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or torch.bfloat16, device=dev)
    elif out.device != dev or not out.is_contiguous() or tuple(out.shape) != shape:
        raise ValueError(f"out must be a contiguous {shape} tensor on the inputs' device")
    _dtype(out, "out", torch.bfloat16, torch.float32)
    return out


def _space(nbytes, dev, torch):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def affine_lora(w, scales, biases, x, lora_a, lora_b, ids, *, bits: int, group_size: int,
                scaling=None, out=None, out_dtype=None, stream=None):
    """y[m] = W x[m] + scaling[a] * lora_b[a] @ (lora_a[a] @ x[m]), a = ids[m]:
    the affine-quantized projection of many requests' tokens, each with its own
    low-rank adapter.

    w, scales, biases, x, bits, group_size, out, out_dtype: as `affine`;
    lora_a [L][R][K] and lora_b [L][N][R]: bf16 or fp16, ranks below R padded
    with zeros; ids: int32 [M], a value outside [0, L) means no adapter;
    scaling: fp32 [L], default 1.  Everything is added in fp32 and rounded once; each
    row is bit-identical to a call with that row alone.
    """
    import torch
    L_ = _lib or _load()
    squeeze = x.dim() == 1
    if squeeze:
        x = x.unsqueeze(0)
    if x.dim() != 2 or w.dim() != 2 or lora_a.dim() != 3:
        raise ValueError("x must be [M][K] (or [K]), w [N][K*bits/32] and lora_a [L][R][K]")
    M, K = x.shape
    N = w.shape[0]
    L, R = lora_a.shape[0], lora_a.shape[1]
    _dtype(x, "x", torch.bfloat16, torch.float32)
    _matrix(w, scales, biases, (N,), K, bits, group_size, "w")
    _dtype(lora_a, "lora_a", torch.bfloat16, torch.float16)
    if lora_b.dtype != lora_a.dtype:
        raise TypeError("lora_a and lora_b must share a dtype")
    _shape(lora_a, "lora_a", L, R, K)
    _shape(lora_b, "lora_b", L, N, R)
    _dtype(ids, "ids", torch.int32)
    _shape(ids, "ids", M)
    named = [(w, "w"), (scales, "scales"), (biases, "biases"), (x, "x"), (lora_a, "lora_a"), (lora_b, "lora_b"), (ids, "ids")]
    if scaling is not None:
        _dtype(scaling, "scaling", torch.float32)
        _shape(scaling, "scaling", L)
        named.append((scaling, "scaling"))
    qmv._check_tensors(named)
    dev = x.device
    with _On(dev, stream, [t for t, _ in named] + [out]) as st:
        out = _out(out, out_dtype, (M, N), dev, torch)
        if M == 0:
            return out
        nbytes = L_.qmv_affine_lora_workspace(M, K, R)
        ws = _space(max(nbytes, 0), dev, torch)
        status = L_.qmv_affine_lora(
            w.data_ptr(), scales.data_ptr(), biases.data_ptr(), x.data_ptr(), out.data_ptr(), lora_a.data_ptr(),
            lora_b.data_ptr(), ids.data_ptr(), None if scaling is None else scaling.data_ptr(), ws.data_ptr(), nbytes,
            M, N, K, bits, group_size, L, R, _DT[x.dtype], _DT[scales.dtype], _DT[out.dtype], _DT[lora_a.dtype], st)
    if status != 0:
        raise QmvError(status, "qmv_affine_lora")
    return out[0] if squeeze else out
