"""The operators beside the quantized product: the adapted projection, the
mixture-of-experts layer and the verification of drafted tokens (include/qmv_ops.h);
norms and rotation of queries and keys, a cache in pages and attention over it
(include/qmv_attn.h).

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


class Cache(ctypes.Structure):
    """qmv_cache, for calls with raw pointers."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v")] + \
               [(n, ctypes.c_longlong) for n in ("k_page", "k_slot", "k_head", "v_page", "v_slot", "v_head")] + \
               [(n, ctypes.c_void_p) for n in ("pages", "starts", "lengths")] + [("pages_row", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("n_pages", "page_size", "n_seqs", "max_pages", "heads", "head_size", "dt")]


class Rotation(ctypes.Structure):
    """qmv_rotation, for calls with raw pointers."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("freqs", "positions", "axes", "q_weight", "k_weight")] + \
               [("positions_row", ctypes.c_longlong), ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int) for n in ("rot", "n_axes", "interleaved", "w_dt")]


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
        R, C = ctypes.POINTER(Rotation), ctypes.POINTER(Cache)
        for name, args, r in (("qmv_rotate", [R] + [P] * 4 + [I] * 4 + [Q] * 4 + [I] * 2 + [P], I),
                              ("qmv_append", [R, C] + [P] * 4 + [I] * 2 + [Q] * 6 + [I, P], I),
                              ("qmv_attend_workspace", [C] + [I] * 6, Q),
                              ("qmv_attend", [C] + [P] * 3 + [Q] + [I] * 2 + [Q] * 2 + [I] * 4 + [ctypes.c_float, I, P], I)):
            f = getattr(L, name)
            f.argtypes, f.restype = args, r
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


def rotate(q, k, freqs, positions, *, axes=None, q_weight=None, k_weight=None, eps: float = 1e-6,
           interleaved: bool = False, out_dtype=None, stream=None):
    """(q, k) with each head normed and turned to its token's position.

    q: bf16 or fp32 [T][heads][D], k: the same with its own heads, each head's values
    contiguous, at any stride (views of one projection's output) that is a multiple of 8;
    D a multiple of 8 up to 256.  q_weight, k_weight: bf16 or fp32 [D], the weights of
    x / sqrt(mean(x^2) + eps), None for no norm.  freqs: fp32 [R / 2], R <= D a multiple
    of 8: pair i is turned by positions * freqs[i], computed in fp64 (None: no rotation).  A
    pair is the values i and i + R / 2, or 2i and 2i + 1 if `interleaved`; values from R on
    stay.  positions: int32 [T], or [A][T] for A axes (time, height, width), where axes, int32
    [R / 2], tells each pair's axis (outside [0, A): not turned).  Outputs: out_dtype,
    bf16 (default) or fp16, rounded once.
    """
    f = (_py or _binding()).rotate
    args = (q, k, freqs, positions, axes, q_weight, k_weight, eps, interleaved, out_dtype)
    return f(*args) if stream is None else _on(stream, f, args[:7], *args)


def append(q, k, v, freqs, k_cache, v_cache, pages, starts, lengths, *, positions=None, axes=None, q_weight=None,
           k_weight=None, eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """`rotate` for the new tokens of a cache's sequences: returns q, and writes keys and
    values to their places in the cache.

    k_cache, v_cache: bf16 or fp16 [pages][page_size][heads][D] in any order of strides;
    pages: int32 [B][n], place j of sequence b is slot j % page_size of page
    pages[b][j // page_size] (a page outside the cache holds nothing); starts: int32 [B + 1],
    tokens starts[b] .. starts[b + 1] - 1 are sequence b's new ones; lengths: int32 [B], its
    places with them.  positions: default each token's place; the rest as `rotate`.  The
    returned q has the cache's dtype.  Rows of tokens that are in no sequence are left as they
    were; places below 0 are not written.  A length above the n * page_size places of the
    table counts as that: the new tokens are then the table's last places, and write over them.
    """
    f = (_py or _binding()).append
    args = (q, k, v, freqs, positions, axes, q_weight, k_weight, eps, interleaved, k_cache, v_cache, pages, starts, lengths, out)
    return f(*args) if stream is None else _on(stream, f, args[:8] + args[10:], *args)


def attend(q, k_cache, v_cache, pages, starts, lengths, *, window: int = 0, sinks: int = 0, scale=None, max_new=None,
           max_length=None, out=None, out_dtype=None, stream=None):
    """[T][heads][D]: attention of each sequence's new tokens over its places in the cache.

    q: the cache's dtype, [T][heads][D] at any stride that is a multiple of 8, heads a
    multiple of the cache's; k_cache .. lengths: as `append`.  New token i of sequence b is
    its place p = lengths[b] - (new tokens of b) + i, and sees place j if j <= p and, with a
    window, j > p - window or j < sinks.  A token that sees nothing gets zeros; what a token
    does not see does not touch its output, NaN included.  scale: default 1 / sqrt(D).
    max_new, max_length: how many new tokens and places a sequence has at most, where the
    program knows; defaults T and what the table holds (the bounds set the sizes of launch and
    scratch memory, and what is above them is left out).  out, out_dtype: as `affine`, bf16 or
    fp32; rows of tokens that are in no sequence are left as they were.  A sequence's up to 16 new
    tokens get the bits that a call for each of them gives.
    """
    f = (_py or _binding()).attend
    args = (q, k_cache, v_cache, pages, starts, lengths, window, sinks, scale, max_new, max_length, out, out_dtype)
    return f(*args) if stream is None else _on(stream, f, args[:6] + (out,), *args)
