"""The operators' C ABI: every declared function is exported, and bad
arguments are refused on the host, before any HIP call (no GPU needed); the
binding's own checks."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qmv_ops.h")
NAMES = ["qmv_affine_lora", "qmv_affine_lora_workspace", "qmv_experts", "qmv_experts_workspace", "qmv_moe",
         "qmv_moe_workspace", "qmv_route", "qmv_route_workspace", "qmv_verify", "qmv_verify_workspace"]


@pytest.fixture(scope="module")
def L():
    from bit_quantized_gemv_amd import ops, qmv
    if not os.path.exists(qmv.library_path()):
        from bit_quantized_gemv_amd import build
        build.build()
    return ops._load()


def test_declared_and_exported(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(qmv_[a-z0-9_]+)\s*\(", src))) == NAMES
    for n in NAMES:
        assert hasattr(L, n), n


def test_status_strings():
    from bit_quantized_gemv_amd import qmv
    for i, n in enumerate(["QMV_E_RANK", "QMV_E_EXPERTS", "QMV_E_WORKSPACE", "QMV_E_VOCAB", "QMV_E_STRIDE"], 11):
        assert qmv.status_string(i) == n
        assert re.search(rf"\b{n}\s*=\s*{i}\b", open(HEADER).read())


# fake, aligned, far-apart addresses: the checks fail before any use
def at(i):
    return (1 << 20) + (i << 40)


LORA = dict(w=at(0), s=at(1), b=at(2), x=at(3), y=at(4), la=at(5), lb=at(6), ids=at(7), scaling=at(8), ws=at(9), nws=1 << 30,
            M=3, N=256, K=512, bits=4, gs=64, L=2, R=16, xdt=2, sdt=2, ydt=2, adt=2)


@pytest.mark.parametrize("kw,code", [
    *[({n: 0}, 1) for n in ("w", "s", "b", "x", "y", "la", "lb", "ids", "ws")],
    (dict(bits=3), 2), (dict(gs=32), 3), (dict(N=0), 4), (dict(K=96), 4), (dict(K=0), 4), (dict(K=(1 << 20) + 64), 4),
    (dict(M=0), 5), (dict(M=65537), 5), (dict(M=-1), 5),
    (dict(w=at(0) + 8), 6), (dict(x=at(3) + 2), 6), (dict(la=at(5) + 8), 6), (dict(ids=at(7) + 2), 6),
    (dict(scaling=at(8) + 1), 6), (dict(ws=at(9) + 4), 6), (dict(y=at(4) + 1), 6),
    (dict(xdt=1), 7), (dict(sdt=0), 7), (dict(ydt=1), 7), (dict(adt=0), 7), (dict(adt=9), 7),
    (dict(y=at(3)), 9), (dict(ws=at(0) + 64), 9), (dict(ws=at(4)), 9), (dict(y=at(6)), 9),
    (dict(R=0), 11), (dict(R=513), 11), (dict(L=0), 11), (dict(L=65537), 11), (dict(nws=0), 13), (dict(nws=100), 13),
])
def test_lora_refuses(L, kw, code):
    a = {**LORA, **kw}
    assert L.qmv_affine_lora(*[a[n] for n in ("w", "s", "b", "x", "y", "la", "lb", "ids", "scaling", "ws", "nws", "M", "N", "K",
                                              "bits", "gs", "L", "R", "xdt", "sdt", "ydt", "adt")], None) == code


MOE = dict(x=at(0), router=at(1), w13=at(2), s13=at(3), b13=at(4), w2=at(5), s2=at(6), b2=at(7), y=at(8), weights=at(9),
           ids=at(10), ws=at(11), nws=1 << 30, T=3, D=512, F=256, E=8, k=2, renorm=1, bits=4, gs=64, xdt=2, rdt=2, sdt=2, ydt=2)
BAD_MOE = [
    (dict(bits=5), 2), (dict(gs=256), 3), (dict(D=96), 4), (dict(F=32), 4), (dict(F=0), 4), (dict(T=0), 5), (dict(T=65537), 5),
    (dict(x=at(0) + 2), 6), (dict(w13=at(2) + 4), 6), (dict(b2=at(7) + 2), 6), (dict(y=at(8) + 1), 6), (dict(ids=at(10) + 1), 6),
    (dict(xdt=1), 7), (dict(sdt=0), 7), (dict(ydt=1), 7), (dict(y=at(0)), 9), (dict(ws=at(5)), 9),
    (dict(E=0), 12), (dict(E=1025), 12), (dict(k=0), 12), (dict(k=33), 12), (dict(nws=64), 13)]


@pytest.mark.parametrize("kw,code", BAD_MOE + [({n: 0}, 1) for n in MOE if MOE[n] >= 1 << 20 and n != "nws"]
                         + [(dict(k=9), 12), (dict(rdt=1), 7), (dict(weights=at(10)), 9)])
def test_moe_refuses(L, kw, code):
    a = {**MOE, **kw}
    assert L.qmv_moe(*[a[n] for n in ("x", "router", "w13", "s13", "b13", "w2", "s2", "b2", "y", "weights", "ids", "ws", "nws",
                                      "T", "D", "F", "E", "k", "renorm", "bits", "gs", "xdt", "rdt", "sdt", "ydt")], None) == code


@pytest.mark.parametrize("kw,code", BAD_MOE + [(dict(weights=0), 1), (dict(ids=0), 1), (dict(y=at(10)), 9)])
def test_experts_refuses(L, kw, code):
    a = {**MOE, **kw}
    assert L.qmv_experts(*[a[n] for n in ("x", "weights", "ids", "w13", "s13", "b13", "w2", "s2", "b2", "y", "ws", "nws", "T", "D",
                                          "F", "E", "k", "bits", "gs", "xdt", "sdt", "ydt")], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), 1), (dict(router=0), 1), (dict(T=0), 5), (dict(D=4), 4), (dict(D=12), 4), (dict(E=0), 12), (dict(E=2000), 12),
    (dict(k=9), 12), (dict(k=0), 12), (dict(xdt=1), 7), (dict(rdt=3), 7), (dict(x=at(0) + 4), 6), (dict(weights=at(0)), 9),
    (dict(nws=1), 13)])
def test_route_refuses(L, kw, code):
    a = {**MOE, **kw}
    assert L.qmv_route(*[a[n] for n in ("x", "router", "weights", "ids", "ws", "nws", "T", "D", "E", "k", "renorm", "xdt", "rdt")],
                       None) == code


VERIFY = dict(l=at(0), d=at(1), u=at(2), q=at(3), t=at(4), n=at(5), tok=at(6), acc=at(7), ws=at(8), nws=1 << 30, B=2, S=3, V=1000,
              lb=4000, lr=1000, qb=3000, qr=1000, ldt=2, qdt=0)


@pytest.mark.parametrize("kw,code", [
    *[({n: 0}, 1) for n in ("l", "d", "u", "tok", "acc", "ws")],
    (dict(l=at(0) + 1), 6), (dict(q=at(3) + 2), 6), (dict(d=at(1) + 2), 6), (dict(t=at(4) + 2), 6), (dict(ws=at(8) + 8), 6),
    (dict(ldt=1), 7), (dict(qdt=1), 7), (dict(tok=at(0)), 9), (dict(ws=at(3)), 9), (dict(acc=at(6)), 9),
    (dict(nws=10), 13), (dict(B=0), 14), (dict(S=-1), 14), (dict(S=256), 14), (dict(V=0), 14), (dict(V=(1 << 26) + 1), 14),
    (dict(B=65536), 14), (dict(lr=-1), 15), (dict(lb=(1 << 40) + 1), 15), (dict(qb=-5), 15)])
def test_verify_refuses(L, kw, code):
    a = {**VERIFY, **kw}
    assert L.qmv_verify(*[a[n] for n in ("l", "d", "u", "q", "t", "n", "tok", "acc", "ws", "nws", "B", "S", "V", "lb", "lr", "qb",
                                         "qr", "ldt", "qdt")], None) == code


def test_workspaces(L):
    assert L.qmv_affine_lora_workspace(1, 512, 5) >= 512 * 2 + 32 * 4          # packed activations, padded ranks
    assert L.qmv_affine_lora_workspace(65536, 512, 32) == L.qmv_affine_lora_workspace(4096, 512, 32)   # taken in pieces
    for bad in ((0, 512, 5), (1, 0, 5), (1, 512, 0), (1, 512, 513)):
        assert L.qmv_affine_lora_workspace(*bad) == -1
    assert L.qmv_moe_workspace(4, 512, 256, 8, 2) >= max(L.qmv_route_workspace(4, 512, 8), L.qmv_experts_workspace(4, 512, 256, 2))
    assert L.qmv_moe_workspace(4, 512, 256, 0, 2) == -1 and L.qmv_experts_workspace(4, 512, 256, 33) == -1
    assert L.qmv_verify_workspace(1, 256, 10) == -1 and L.qmv_verify_workspace(2, 3, 1000) > 0


def tensors(op):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    if op == "lora":
        return dict(w=i(8, 16), scales=z(8, 2), biases=z(8, 2), x=z(3, 128), lora_a=z(2, 4, 128), lora_b=z(2, 8, 4), ids=i(3),
                    bits=4, group_size=64)
    if op == "moe":
        return dict(x=z(3, 128), router=z(4, 128), gate_up=(i(4, 128, 16), z(4, 128, 2), z(4, 128, 2)),
                    down=(i(4, 128, 8), z(4, 128, 1), z(4, 128, 1)), top_k=2, bits=4, group_size=64)
    return dict(logits=z(2, 4, 10), draft=i(2, 3), uniforms=z(2, 4, dt=torch.float32))


@pytest.mark.parametrize("op,kw,error,text", [
    ("lora", dict(x=torch.zeros(3, 128, dtype=torch.float16)), TypeError, "x must be bfloat16 or float32"),
    ("lora", dict(x=torch.zeros(3, 192).bfloat16()), ValueError, "w has shape"),
    ("lora", dict(lora_b=torch.zeros(2, 9, 4).bfloat16()), ValueError, "lora_b has shape"),
    ("lora", dict(lora_b=torch.zeros(2, 8, 4).half()), TypeError, "share a dtype"),
    ("lora", dict(ids=torch.zeros(3)), TypeError, "ids must be int32"),
    ("lora", dict(ids=torch.zeros(2).int()), ValueError, "ids has shape"),
    ("lora", dict(scaling=torch.zeros(3)), ValueError, "scaling has shape"),
    ("lora", dict(bits=3), ValueError, "bits"), ("lora", dict(group_size=32), ValueError, "group_size"),
    ("lora", {}, ValueError, "CUDA"),
    ("moe", dict(top_k=5), ValueError, "top_k"), ("moe", dict(top_k=0), ValueError, "top_k"),
    ("moe", dict(router=torch.zeros(4, 64)), ValueError, "router must be"),
    ("moe", dict(router=torch.zeros(5, 128)), ValueError, "gate_up has shape"),
    ("moe", dict(x=torch.zeros(128)), ValueError, "x must be"),
    ("moe", {}, ValueError, "CUDA"),
    ("verify", dict(logits=torch.zeros(2, 4, 10).half()), TypeError, "logits must be"),
    ("verify", dict(draft=torch.zeros(2, 3).long()), TypeError, "draft must be int32"),
    ("verify", dict(draft=torch.zeros(2, 4).int()), ValueError, "draft has shape"),
    ("verify", dict(uniforms=torch.zeros(2, 3)), ValueError, "uniforms has shape"),
    ("verify", dict(draft_probs=torch.zeros(2, 3, 9)), ValueError, "draft_probs has shape"),
    ("verify", dict(lengths=torch.zeros(2)), TypeError, "lengths must be int32"),
    ("verify", dict(temperature=torch.zeros(3)), ValueError, "temperature has shape"),
    ("verify", {}, ValueError, "CUDA"),
])
def test_binding_refuses(L, op, kw, error, text):
    import bit_quantized_gemv_amd as q
    f = {"lora": q.affine_lora, "moe": q.moe, "verify": q.verify}[op]
    with pytest.raises(error, match=text):
        f(**{**tensors(op), **kw})
