"""The operators beside the quantized product (include/qmv_ops.h): the adapted
projection, the mixture-of-experts layer and the verification of drafted tokens.

Each is one call of the compiled binding (csrc/ops_py.cpp), which checks the
arguments, allocates outputs and scratch memory on the stream that the call runs
on and calls the C ABI.  Every step runs in the HIP kernels of lib/libqmv.so, and
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

from . import qmv
from .qmv import QmvError

_PY_PATH = os.path.join(os.path.dirname(qmv.library_path()), "qmv_ops_py.so")
_lib = None
_py = None


def _load():
    """The C ABI, for calls with raw pointers."""
    global _lib
    if _lib is None:
        L = qmv.lib()
        P, I, Q = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        for name, args in (("qmv_affine_lora", [P] * 10 + [Q] + [I] * 11 + [P]),
                           ("qmv_route", [P] * 5 + [Q] + [I] * 7 + [P]),
                           ("qmv_experts", [P] * 11 + [Q] + [I] * 10 + [P]),
                           ("qmv_moe", [P] * 12 + [Q] + [I] * 12 + [P]),
                           ("qmv_verify", [P] * 9 + [Q] + [I] * 3 + [Q] * 4 + [I] * 2 + [P])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, I
        for name, n in (("qmv_affine_lora_workspace", 3), ("qmv_route_workspace", 3), ("qmv_experts_workspace", 4),
                        ("qmv_moe_workspace", 5), ("qmv_verify_workspace", 3)):
            f = getattr(L, name)
            f.argtypes, f.restype = [I] * n, Q
        _lib = L
    return _lib


def _binding():
    global _py
    if _py is None:
        import importlib.util
        import torch  # noqa: F401  (its libraries first)
        if not os.path.exists(_PY_PATH):
            raise RuntimeError(f"{_PY_PATH} is not built; run __graft_entry__.build()")
        qmv.lib()
        spec = importlib.util.spec_from_file_location("qmv_ops_py", _PY_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.set_error(QmvError)
        _py = m
    return _py


def _on(stream, f, tensors, *args):
    """The call on another stream than the current one.  The inputs are recorded
    on it, so that their memory is not handed out again before the call has read it."""
    import torch
    tensors = [t for t in tensors if t is not None]
    dev = tensors[0].device
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the inputs on {dev}")
    if stream != torch.cuda.current_stream(dev):
        for t in tensors:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return f(*args)


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
    f = (_py or _binding()).affine_lora
    args = (w, scales, biases, x, lora_a, lora_b, ids, scaling, bits, group_size, out, out_dtype)
    return f(*args) if stream is None else _on(stream, f, args[:8] + (out,), *args)


def route(x, router, *, top_k: int, renormalize: bool = True, stream=None):
    """(weights, ids) of a mixture-of-experts router: the top_k largest products
    x[t] . router[e] of every token in descending order (ties to the lowest expert;
    computed in fp64) and their softmax, over the chosen experts if `renormalize`, else
    over all.

    x: bf16 or fp32 [T][D]; router: bf16 or fp32 [E][D], D a multiple of 8;
    weights: fp32 [T][top_k]; ids: int32 [T][top_k].
    """
    f = (_py or _binding()).route
    args = (x, router, top_k, renormalize)
    return f(*args) if stream is None else _on(stream, f, args[:2], *args)


def experts(x, weights, ids, gate_up, down, *, bits: int, group_size: int, out=None, out_dtype=None, stream=None):
    """y[t] = sum over j of weights[t][j] * Down_e(silu(Gate_e x[t]) * Up_e x[t]),
    e = ids[t][j]: the chosen affine-quantized experts of every token.

    x: bf16 or fp32 [T][D]; weights: fp32 [T][k]; ids: int32 [T][k], a value
    outside [0, E) is an empty slot; gate_up: (codes [E][2F][D*bits/32], scales, biases
    [E][2F][D/group_size]), F gate rows before F up rows; down: (codes
    [E][D][F*bits/32], scales, biases [E][D][F/group_size]); out, out_dtype: as
    `affine`.  Everything between is fp32 and y is rounded once; each token is
    bit-identical to a call with that token alone.
    """
    f = (_py or _binding()).experts
    args = (x, weights, ids, *gate_up, *down, bits, group_size, out, out_dtype)
    return f(*args) if stream is None else _on(stream, f, args[:9] + (out,), *args)


def moe(x, router, gate_up, down, *, top_k: int, bits: int, group_size: int, renormalize: bool = True,
        out=None, out_dtype=None, return_routing: bool = False, stream=None):
    """A whole mixture-of-experts layer: `route`, then `experts` on what it
    chose.  Returns y [T][D], or (y, weights, ids) with return_routing."""
    f = (_py or _binding()).moe
    args = (x, router, *gate_up, *down, top_k, renormalize, bits, group_size, out, out_dtype)
    r = f(*args) if stream is None else _on(stream, f, args[:8] + (out,), *args)
    return r if return_routing else r[0]


def verify(logits, draft, uniforms, *, draft_probs=None, temperature=None, lengths=None, stream=None):
    """(tokens, accepted): drafted tokens accepted or replaced so that what is
    emitted follows the target's distribution p = softmax(logits / temperature).

    logits: bf16 or fp32 [B][S+1][V], rows of contiguous values at any stride; draft: int32
    [B][S]; uniforms: fp32 [B][S+1] in [0, 1); draft_probs: the drafter's probabilities q,
    bf16 or fp32 [B][S][V], or None for a drafter that gives tokens only (q is 1 at the
    drafted token); temperature: fp32 [B], not above 0 for greedy, default 1;
    lengths: int32 [B], how many of a request's S tokens are drafted, default all.

    Position j < lengths[b] is accepted while uniforms[b][j] * q(x_j) < p(x_j).  The first
    that is not gets a token sampled from max(p - q, 0) (from p if nothing is left of it); if
    all are accepted, the position after them gets one sampled from p.  Samples
    are the lowest index whose prefix sum passes uniforms[b][lengths[b]] times the total.  All
    decisions are those of fp64 sums.  NaN and -inf logits have probability 0; a row with nothing
    else rejects its position and gives the token -1.

    tokens: int32 [B][S+1], the accepted tokens, the sampled one, then -1; accepted: int32 [B].
    """
    f = (_py or _binding()).verify
    args = (logits, draft, uniforms, draft_probs, temperature, lengths)
    return f(*args) if stream is None else _on(stream, f, args, *args)
