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


def _tokens(x):
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [T][D]")
    _dtype(x, "x", torch.bfloat16, torch.float32)
    return x.shape


def _router(x, router, top_k):
    import torch
    _dtype(router, "router", torch.bfloat16, torch.float32)
    if router.dim() != 2 or router.shape[1] != x.shape[1]:
        raise ValueError(f"router must be [E][{x.shape[1]}], got {tuple(router.shape)}")
    E = router.shape[0]
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be in [1, {E}], got {top_k}")
    return E


def _expert_weights(gate_up, down, E, D, bits, gs):
    w13, s13, b13 = gate_up
    w2, s2, b2 = down
    if w13.dim() != 3 or w13.shape[1] % 2 != 0:
        raise ValueError("the gate and up codes must be [E][2F][D*bits/32]")
    E = w13.shape[0] if E is None else E
    F = w13.shape[1] // 2
    _matrix(w13, s13, b13, (E, 2 * F), D, bits, gs, "gate_up")
    _matrix(w2, s2, b2, (E, D), F, bits, gs, "down")
    if s2.dtype != s13.dtype:
        raise TypeError("the two products' scales must share a dtype")
    return E, F, [(w13, "gate_up"), (s13, "gate_up scales"), (b13, "gate_up biases"), (w2, "down"), (s2, "down scales"),
                  (b2, "down biases")]


def route(x, router, *, top_k: int, renormalize: bool = True, stream=None):
    """(weights, ids) of a mixture-of-experts router: the top_k largest products
    x[t] . router[e] of every token in descending order (ties to the lowest expert;
    computed in fp64) and their softmax, over the chosen experts if `renormalize`, else
    over all.

    x: bf16 or fp32 [T][D]; router: bf16 or fp32 [E][D], D a multiple of 8;
    weights: fp32 [T][top_k]; ids: int32 [T][top_k].
    """
    import torch
    L_ = _lib or _load()
    T, D = _tokens(x)
    E = _router(x, router, top_k)
    qmv._check_tensors(((x, "x"), (router, "router")))
    dev = x.device
    with _On(dev, stream, (x, router)) as st:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        if T == 0:
            return weights, ids
        nbytes = L_.qmv_route_workspace(T, D, E)
        ws = _space(max(nbytes, 0), dev, torch)
        status = L_.qmv_route(x.data_ptr(), router.data_ptr(), weights.data_ptr(), ids.data_ptr(), ws.data_ptr(), nbytes,
                              T, D, E, top_k, renormalize, _DT[x.dtype], _DT[router.dtype], st)
    if status != 0:
        raise QmvError(status, "qmv_route")
    return weights, ids


def experts(x, weights, ids, gate_up, down, *, bits: int, group_size: int, out=None, out_dtype=None, stream=None):
    """y[t] = sum over j of weights[t][j] * Down_e(silu(Gate_e x[t]) * Up_e x[t]),
    e = ids[t][j]: the chosen affine-quantized experts of every token.

    x: bf16 or fp32 [T][D]; weights: fp32 [T][k]; ids: int32 [T][k], a value
    outside [0, E) is an empty slot; gate_up: (codes [E][2F][D*bits/32], scales, biases
    [E][2F][D/group_size]), F gate rows before F up rows; down: (codes
    [E][D][F*bits/32], scales, biases [E][D][F/group_size]); out, out_dtype: as
    `affine`.  Everything between is fp32; each token is bit-identical to a call with
    that token alone.
    """
    import torch
    L_ = _lib or _load()
    T, D = _tokens(x)
    E, F, mats = _expert_weights(gate_up, down, None, D, bits, group_size)
    _dtype(weights, "weights", torch.float32)
    _dtype(ids, "ids", torch.int32)
    if ids.dim() != 2:
        raise ValueError("ids must be [T][k]")
    k = ids.shape[1]
    _shape(ids, "ids", T, k)
    _shape(weights, "weights", T, k)
    named = [(x, "x"), (weights, "weights"), (ids, "ids")] + mats
    qmv._check_tensors(named)
    dev = x.device
    with _On(dev, stream, [t for t, _ in named] + [out]) as st:
        out = _out(out, out_dtype, (T, D), dev, torch)
        if T == 0:
            return out
        nbytes = L_.qmv_experts_workspace(T, D, F, k)
        ws = _space(max(nbytes, 0), dev, torch)
        status = L_.qmv_experts(x.data_ptr(), weights.data_ptr(), ids.data_ptr(), *[t.data_ptr() for t, _ in mats],
                                out.data_ptr(), ws.data_ptr(), nbytes, T, D, F, E, k, bits, group_size,
                                _DT[x.dtype], _DT[mats[1][0].dtype], _DT[out.dtype], st)
    if status != 0:
        raise QmvError(status, "qmv_experts")
    return out


def moe(x, router, gate_up, down, *, top_k: int, bits: int, group_size: int, renormalize: bool = True,
        out=None, out_dtype=None, return_routing: bool = False, stream=None):
    """A whole mixture-of-experts layer: `route`, then `experts` on what it
    chose.  Returns y [T][D], or (y, weights, ids) with return_routing."""
    import torch
    L_ = _lib or _load()
    T, D = _tokens(x)
    E = _router(x, router, top_k)
    E, F, mats = _expert_weights(gate_up, down, E, D, bits, group_size)
    named = [(x, "x"), (router, "router")] + mats
    qmv._check_tensors(named)
    dev = x.device
    with _On(dev, stream, [t for t, _ in named] + [out]) as st:
        out = _out(out, out_dtype, (T, D), dev, torch)
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        status = 0
        if T != 0:
            nbytes = L_.qmv_moe_workspace(T, D, F, E, top_k)
            ws = _space(max(nbytes, 0), dev, torch)
            status = L_.qmv_moe(x.data_ptr(), router.data_ptr(), *[t.data_ptr() for t, _ in mats], out.data_ptr(),
                                weights.data_ptr(), ids.data_ptr(), ws.data_ptr(), nbytes, T, D, F, E, top_k,
                                renormalize, bits, group_size, _DT[x.dtype], _DT[router.dtype],
                                _DT[mats[1][0].dtype], _DT[out.dtype], st)
    if status != 0:
        raise QmvError(status, "qmv_moe")
    return (out, weights, ids) if return_routing else out


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
    are the lowest index whose prefix sum passes uniforms[b][lengths[b]] times the total, in
    fp64; the sums behind an accept decision are within 2^-20 of their value.  NaN and -inf logits have probability 0; a row with nothing else rejects its
    position and gives the token -1.

    tokens: int32 [B][S+1], the accepted tokens, the sampled one, then -1; accepted: int32 [B].
    """
    import torch
    L_ = _lib or _load()
    if logits.dim() != 3 or logits.shape[1] < 1:
        raise ValueError("logits must be [B][S+1][V]")
    B, S1, V = logits.shape
    S = S1 - 1
    _dtype(logits, "logits", torch.bfloat16, torch.float32)
    _dtype(draft, "draft", torch.int32)
    _shape(draft, "draft", B, S)
    _dtype(uniforms, "uniforms", torch.float32)
    _shape(uniforms, "uniforms", B, S1)
    named = [(draft, "draft"), (uniforms, "uniforms")]
    rows = [(logits, "logits")]
    if draft_probs is not None:
        _dtype(draft_probs, "draft_probs", torch.bfloat16, torch.float32)
        _shape(draft_probs, "draft_probs", B, S, V)
        rows.append((draft_probs, "draft_probs"))
    if temperature is not None:
        _dtype(temperature, "temperature", torch.float32)
        _shape(temperature, "temperature", B)
        named.append((temperature, "temperature"))
    if lengths is not None:
        _dtype(lengths, "lengths", torch.int32)
        _shape(lengths, "lengths", B)
        named.append((lengths, "lengths"))
    dev = logits.device
    for t, n in rows:
        if not t.is_cuda:
            raise ValueError(f"{n} must be a CUDA (HIP) tensor")
        if t.device != dev:
            raise ValueError(f"{n} is on {t.device}, the other inputs on {dev}")
        if V > 1 and t.stride(2) != 1:
            raise ValueError(f"{n}: the values of a row must be contiguous")
    qmv._check_tensors(named)
    if draft.device != dev:
        raise ValueError(f"draft is on {draft.device}, the other inputs on {dev}")
    with _On(dev, stream, [t for t, _ in named + rows]) as st:
        tokens = torch.empty((B, S1), dtype=torch.int32, device=dev)
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
        if B == 0:
            return tokens, accepted
        nbytes = L_.qmv_verify_workspace(B, S, V)
        ws = _space(max(nbytes, 0), dev, torch)
        q = draft_probs if S > 0 else None
        status = L_.qmv_verify(
            logits.data_ptr(), draft.data_ptr(), uniforms.data_ptr(), None if q is None else q.data_ptr(),
            None if temperature is None else temperature.data_ptr(), None if lengths is None else lengths.data_ptr(),
            tokens.data_ptr(), accepted.data_ptr(), ws.data_ptr(), nbytes, B, S, V, logits.stride(0), logits.stride(1),
            0 if q is None else q.stride(0), 0 if q is None else q.stride(1), _DT[logits.dtype],
            DT_F32 if q is None else _DT[q.dtype], st)
    if status != 0:
        raise QmvError(status, "qmv_verify")
    return tokens, accepted
